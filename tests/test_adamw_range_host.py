"""lstm_adamw_step: hyperparameters that are numbers in float64 but not in the float32 the kernel computes in (CPU).

An eps that rounds to 0, or to a float32 below the normal range (its reciprocal is infinite), gives 0 / 0 where
gradient and moments are zero; a step size or a decay that rounds to infinity gives infinity times 0.
"""
import pytest

from layer_lstm_b200 import binding
from test_adamw_host import _step


@pytest.mark.parametrize("kw", [dict(eps=1e-50), dict(eps=1e-46), dict(eps=1e-40), dict(eps=1.1e-38), dict(eps=1e38),
                                dict(eps=1e39), dict(eps=float("nan")), dict(lr=1e39), dict(lr=1e38, beta1=0.9),
                                dict(lr=1e30, weight_decay=1e10), dict(lr=float("inf")),
                                dict(weight_decay=float("inf"))])
def test_refused_beyond_float32(kw):
    assert _step(binding.make_adamw_desc(1, **kw)) == binding.LSTM_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(eps=2.0 ** -126), dict(eps=2.0 ** 126), dict(eps=1e-30), dict(lr=1e37, beta1=0.9),
                                dict(lr=0.0, weight_decay=1e300), dict(weight_decay=1e30),
                                dict(beta1=1 - 2.0 ** -53, beta2=1 - 2.0 ** -53)])
def test_accepted_at_the_borders(kw):
    # an empty 8-bit read-out looks at the description and enqueues nothing; without a GPU it ends there
    got = binding.lstm_adamw_read_state(binding.make_adamw_desc(0, state_bits=8, **kw), [], [], [], [], [], [], [],
                                        stream=0)
    assert got in (binding.LSTM_OK, binding.LSTM_ERR_CUDA)

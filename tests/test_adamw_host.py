"""lstm_adamw_step / lstm_adamw_read_state: what they refuse, before anything is enqueued (CPU)."""
import ctypes
import re

import pytest
import torch

from layer_lstm_b200 import binding
from test_header_binding import C_SIZES, _header, _struct_fields


def _step(desc, numel=(4,), p=(256,), copy=None, g=(256,), m=(256,), v=(256,), ms=None, vs=None, step=256,
          scalars=None):
    return binding.lstm_adamw_step(desc, list(numel), p and list(p), copy and list(copy), g and list(g),
                                   m and list(m), v and list(v), ms and list(ms), vs and list(vs), step, scalars, 0)


def test_struct_matches_header():
    fields = _struct_fields(_header(), "lstm_adamw_desc")
    assert [n for _, n, _ in fields] == [n for n, _ in binding.lstm_adamw_desc._fields_]
    for (typ, name, _), (_, ptype) in zip(fields, binding.lstm_adamw_desc._fields_):
        assert ctypes.sizeof(ptype) == C_SIZES[typ], name


@pytest.mark.parametrize("kw", [dict(state_bits=16), dict(grad_dtype=3), dict(lr=-1.0), dict(lr=float("nan")),
                                dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=float("nan")),
                                dict(eps=0.0), dict(eps=float("inf")), dict(weight_decay=-0.1),
                                dict(num_tensors=-1)])
def test_refused_descriptions(kw):
    args = dict(num_tensors=1)
    args.update(kw)
    assert _step(binding.make_adamw_desc(**args)) == binding.LSTM_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(numel=(-1,)), dict(p=None), dict(g=None), dict(m=None), dict(v=None),
                                dict(p=(0,)), dict(g=(0,)), dict(m=(0,)), dict(v=(0,)), dict(p=(258,)),
                                dict(g=(257,)), dict(m=(258,)), dict(v=(259,)), dict(copy=(257,)),
                                dict(step=None), dict(step=260), dict(scalars=258)])
def test_refused_pointers(kw):
    assert _step(binding.make_adamw_desc(1), **kw) == binding.LSTM_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(), dict(ms=(256,)), dict(vs=(256,)), dict(ms=(256,), vs=(258,)),
                                dict(ms=(0,), vs=(256,))])
def test_refused_scales(kw):
    assert _step(binding.make_adamw_desc(1, state_bits=8), **kw) == binding.LSTM_ERR_INVALID_ARG


def test_read_state_refuses():
    one = [256]
    for desc, args in ((binding.make_adamw_desc(1), [one] * 6),
                       (binding.make_adamw_desc(1, state_bits=8), [one] * 5 + [None]),
                       (binding.make_adamw_desc(1, state_bits=8), [one] * 4 + [[258], one]),
                       (binding.make_adamw_desc(1, state_bits=8), [one, one, [0], one, one, one])):
        assert binding.lstm_adamw_read_state(desc, [4], *args, stream=0) == binding.LSTM_ERR_INVALID_ARG


def test_optimizer_refuses_tensors():
    from layer_lstm_b200.optim import AdamW
    p, g = torch.zeros(4, 4), torch.zeros(4, 4)
    for bad in (dict(params=[p.double()], grads=[g]), dict(params=[p.t()[:2]], grads=[g[:2]]),
                dict(params=[p], grads=[g.half()]), dict(params=[p], grads=[g[:2]]), dict(params=[p], grads=[]),
                dict(params=[p], grads=[g], copies=[g]), dict(params=[p], grads=[g], state_bits=4),
                dict(params=[p], grads=[g], scalars=torch.zeros(3)),
                dict(params=[p, p], grads=[g, g.bfloat16()])):
        with pytest.raises(ValueError):
            AdamW(**bad)


def test_timing_kind_is_listed():
    names = re.search(r"Kinds \(the suffix.*?\.\n", open(
        __file__.replace("tests/test_adamw_host.py", "include/lstm.h")).read(), flags=re.S).group(0)
    assert "adamw" in names

"""lstm_linear_attention_forward and _backward without the states nobody asked for (GPU): s_n and ds0 NULL.

What is left out is a last state that nothing else reads, so out, dq, dk and dv are those of the calls that do
ask, bit for bit.  Rows and heads enough that every block walks many of them: runs of items whose last chunk
forms no state stand behind one another in a block's pipeline, beside items that do form one.
"""
import pytest
import torch

from layer_lstm_b200 import binding
from test_linear_attention_gpu import _check, _desc, _inputs, _run

pytestmark = pytest.mark.gpu


def _without_states(t, d, dt, ws):
    out = torch.full_like(t["go"], 7.0)
    binding.check(binding.lstm_linear_attention_forward(d, t["q"], t["k"], t["v"], t["ld"], t["s0"], out, None, ws,
                                                        lengths=t["lengths"]))
    assert binding.lstm_query_status(ws) == binding.LSTM_OK
    dq, dk, dv = (torch.full_like(t[x], 7.0) for x in "qkv")
    binding.check(binding.lstm_linear_attention_backward(d, t["q"], t["k"], t["v"], t["ld"], t["s0"], t["go"],
                                                         t["gs"], dq, dk, dv, None, ws, lengths=t["lengths"]))
    assert binding.lstm_query_status(ws) == binding.LSTM_OK
    return [out, dq, dk, dv]


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (128, 64), (64, 128), (48, 80)])
@pytest.mark.parametrize("T", [1, 70, 128, 129, 300])
def test_same_values_without_states(T, dk, dv, dt, cuda_lib):
    B, H = 40, 16
    for ragged in (False, True):
        t = _inputs(B, T, H, dk, dv, dt, T + ragged, ragged)
        if ragged:
            t["lengths"][5:12] = 0
        d = _desc(t, B, T, H, dk, dv, dt)
        want = _run(t, d, dt)
        ws = torch.full((binding.lstm_linear_attention_workspace_size(d),), 255, device="cuda", dtype=torch.uint8)
        for _ in range(3):
            for name, a, b in zip(("out", "dq", "dk", "dv"), (want[0], *want[2:5]),
                                  _without_states(t, d, dt, ws)):
                assert torch.equal(a, b), name


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
@pytest.mark.parametrize("B,T,H", [(2, 300, 2), (1, 1500, 1)])
def test_values_without_states(B, T, H, dk, dv, dt, cuda_lib):
    """The same against the recurrence: whole rows, and rows cut into segments."""
    t = _inputs(B, T, H, dk, dv, dt, 30, True)
    d = _desc(t, B, T, H, dk, dv, dt)
    want = _run(t, d, dt)
    ws = torch.empty(binding.lstm_linear_attention_workspace_size(d), device="cuda", dtype=torch.uint8)
    out, dq, dk_, dv_ = _without_states(t, d, dt, ws)
    _check(t, d, dt, [out, want[1], dq, dk_, dv_, want[5]])

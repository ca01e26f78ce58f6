"""optim.AdamW refuses tensors that share memory a step writes (CPU): a weight given twice, a view of another one,
moments used for two parameters, a gradient in a parameter's place.  Gradients may share memory with one another."""
import pytest
import torch

from layer_lstm_b200.optim import AdamW


def _zeros(*sizes):
    return [torch.zeros(n) for n in sizes]


def _refused(*a, **kw):
    with pytest.raises(ValueError, match="share"):
        AdamW(*a, **kw)


@pytest.mark.parametrize("bits", [32, 8])
def test_refused(bits):
    whole = torch.zeros(600)
    p = torch.zeros(300)
    _refused([p, p], _zeros(300, 300), state_bits=bits)
    _refused([whole[:300], whole[299:599]], _zeros(300, 300), state_bits=bits)
    _refused([whole, whole[10:12]], _zeros(600, 2), state_bits=bits)
    _refused([p], [p], state_bits=bits)
    _refused([whole[:300], torch.zeros(300)], [torch.zeros(300), whole[200:500]], state_bits=bits)
    c = torch.zeros(300, dtype=torch.bfloat16)
    _refused(_zeros(300, 300), _zeros(300, 300), copies=[c, c], state_bits=bits)


@pytest.mark.parametrize("bits", [32, 8])
def test_shared_moments_are_refused(bits):
    opt = AdamW(_zeros(300, 300), _zeros(300, 300), state_bits=bits)
    s = opt.state
    for name in ("m", "v") + (("m_scale", "v_scale") if bits == 8 else ()):
        _refused(_zeros(300, 300), _zeros(300, 300), state_bits=bits, state=dict(s, **{name: [s[name][0]] * 2}))
    if bits == 32:
        _refused(_zeros(300, 300), _zeros(300, 300), state=dict(s, v=s["m"]))


@pytest.mark.parametrize("bits", [32, 8])
def test_neighbours_and_shared_gradients_pass(bits):
    flat = torch.zeros(900)
    g = torch.zeros(300)
    AdamW([flat[:300], flat[300:600], flat[600:]], [g, g, g], state_bits=bits)
    AdamW([flat[:300], torch.zeros(0), torch.zeros(0)], [g, torch.zeros(0), torch.zeros(0)], state_bits=bits)
    AdamW([flat[:300]], [flat[300:600]], state_bits=bits)

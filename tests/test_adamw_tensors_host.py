"""optim.AdamW calls the library with the tensors it holds at the step, not with those of its construction (CPU:
the call is recorded in the place of the library's)."""
import ctypes
import gc
import weakref

import pytest
import torch

from layer_lstm_b200 import binding
from layer_lstm_b200.optim import AdamW


@pytest.fixture
def calls(monkeypatch):
    got = []

    def step(desc, numel, *a):
        *lists, counter, scalars, stream = a
        got.append(dict(n=list(numel), lists=[None if x is None else list(x) for x in lists],
                        step=counter.data_ptr(), desc=(desc.num_tensors, desc.grad_dtype, desc.state_bits)))
        return binding.LSTM_OK

    monkeypatch.setattr(binding, "lstm_adamw_step", step)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)
    return got


def _addresses(opt):
    s = opt.state
    lists = [opt.params, opt.copies, opt.grads, s["m"], s["v"]] + [s["m_scale"], s["v_scale"]]
    return [None if ts is None else [None if t is None else t.data_ptr() for t in ts] for ts in lists]


def _make(bits, n=3):
    p, g = [torch.randn(300 + i) for i in range(n)], [torch.randn(300 + i) for i in range(n)]
    copies = [p[0].bfloat16(), None, p[2].bfloat16()]
    return AdamW(p, g, copies=copies, state_bits=bits)


@pytest.mark.parametrize("bits", [32, 8])
def test_restored_state_is_what_a_step_updates(bits, calls):
    opt = _make(bits)
    opt.step()
    assert calls[-1]["lists"] == _addresses(opt)
    # a whole state, an entry of it, one tensor of an entry, a tensor's storage
    old = opt.state
    opt.state = {k: [t.clone() for t in x] if isinstance(x, list) else x.clone() if x is not None else None
                 for k, x in old.items()}
    opt.step()
    assert calls[-1]["lists"] == _addresses(opt) and calls[-1]["step"] == opt.state["step"].data_ptr()
    opt.state["m"] = [t.clone() for t in opt.state["m"]]
    opt.step()
    assert calls[-1]["lists"] == _addresses(opt)
    opt.state["v"][1] = opt.state["v"][1].clone()
    opt.params[2].data = opt.params[2].data.clone()
    opt.grads[0] = opt.grads[0].clone()
    opt.step()
    assert calls[-1]["lists"] == _addresses(opt)
    # what is replaced may go, what a step was given last stays
    gone = weakref.ref(old["m"][0])
    del old
    gc.collect()
    assert gone() is None


def test_gradient_type_may_change(calls):
    opt = _make(32)
    opt.grads[:] = [g.bfloat16() for g in opt.grads]
    opt.step()
    assert calls[-1]["desc"] == (3, binding.LSTM_BF16, 32) and calls[-1]["lists"] == _addresses(opt)


@pytest.mark.parametrize("bits", [32, 8])
def test_replacements_are_checked(bits, calls):
    def spoil(what):
        opt = _make(bits)
        what(opt)
        with pytest.raises(ValueError):
            opt.step()
        assert not calls

    spoil(lambda o: o.state.__setitem__("m", [t[:10].clone() for t in o.state["m"]]))
    spoil(lambda o: o.state["v"].__setitem__(0, o.state["v"][0].double()))
    spoil(lambda o: o.state.__setitem__("step", torch.zeros(1)))
    spoil(lambda o: o.state["m"].pop())
    spoil(lambda o: o.grads.__setitem__(1, torch.randn(7)))
    spoil(lambda o: o.params.append(torch.randn(7)))
    if bits == 8:
        spoil(lambda o: o.state["m_scale"].__setitem__(0, torch.zeros(1)))


def test_arrays_are_kept_while_the_tensors_are(calls):
    opt = _make(8)
    arrays = opt._ptr
    opt.step()
    opt.params[0].mul_(0.5)
    opt.desc.lr = 0.25
    opt.step()
    assert opt._ptr is arrays and all(x is None or isinstance(x, ctypes.Array) for x in arrays)
    assert calls[0] == calls[1]

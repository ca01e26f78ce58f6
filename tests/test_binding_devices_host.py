"""The operators' calls with addresses and tensors mixed: the call runs on the tensors' device, whichever argument
brings the first one (CPU: stand-ins for tensors, the library's call recorded)."""
import contextlib

import pytest
import torch

from layer_lstm_b200 import binding

F32, I32, U8 = torch.float32, torch.int32, torch.uint8


class Fake:
    """What the binding asks of a tensor, on GPU 1."""

    def __init__(self, *shape, dtype=F32, device=1):
        self.shape, self.dtype, self.dev = shape, dtype, device

    def numel(self):
        return int(torch.Size(self.shape).numel())

    def element_size(self):
        return 4

    def get_device(self):
        return self.dev

    def is_contiguous(self):
        return True

    def dim(self):
        return len(self.shape)

    def data_ptr(self):
        return 4096


class Library:
    def __init__(self):
        self.ran_on = []

    def __getattr__(self, name):
        return lambda *a: self.ran_on.append(torch.cuda.current_device()) or binding.LSTM_OK


@pytest.fixture
def lib(monkeypatch):
    lib, now = Library(), [0]

    @contextlib.contextmanager
    def device(d):
        now[0], old = d, now[0]
        yield
        now[0] = old

    monkeypatch.setattr(binding, "load", lambda: lib)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "device", device)
    return lib


B, T, H, D = 2, 1, 2, 8
X, S, L = (B, T, H, D), (B, H, D, D), (H,)
NORM = binding.make_norm_desc(4, 8)
ATT = binding.make_attention_desc(B, T, H, D, D)
CALLS = {
    "norm_forward": (lambda a: binding.lstm_layer_norm_forward(NORM, *a, stream=0),
                     [(4, 8), (8,), (8,), (4, 8), (4,), (4,)]),
    "norm_backward": (lambda a: binding.lstm_layer_norm_backward(NORM, *a, stream=0, ws_bytes=1),
                      [(4, 8), (4, 8), (8,), (4,), (4,), (4, 8), (8,), (8,), (512,)]),
    "att_forward": (lambda a: binding.lstm_linear_attention_forward(ATT, *a[:-1], stream=0, ws_bytes=1, lengths=a[-1]),
                    [X, X, X, L, S, X, S, (512,), (B,)]),
    "att_backward": (lambda a: binding.lstm_linear_attention_backward(ATT, *a[:-1], stream=0, ws_bytes=1,
                                                                      lengths=a[-1]),
                     [X, X, X, L, S, X, S, X, X, X, S, (512,), (B,)]),
    "att_step": (lambda a: binding.lstm_linear_attention_step(ATT, *a[:-1], stream=0, lengths=a[-1]),
                 [X, X, X, L, S, X, (B,)]),
}


def _fake(name, shapes, i, device=1):
    return Fake(*shapes[i], dtype=I32 if name.startswith("att") and i == len(shapes) - 1 else F32, device=device)


@pytest.mark.parametrize("name", list(CALLS))
def test_one_tensor_among_addresses(name, lib):
    call, shapes = CALLS[name]
    for i in range(len(shapes)):
        a = [256] * len(shapes)
        a[i] = _fake(name, shapes, i)
        assert call(a) == binding.LSTM_OK, i
        assert lib.ran_on.pop() == 1, i


@pytest.mark.parametrize("name", list(CALLS))
def test_tensors_of_two_devices_are_refused(name, lib):
    call, shapes = CALLS[name]
    for i in range(1, len(shapes)):
        for j in range(i):
            a = [256] * len(shapes)
            a[i], a[j] = _fake(name, shapes, i, 1), _fake(name, shapes, j, 0)
            assert call(a) == binding.LSTM_ERR_INVALID_ARG, (i, j)
            a[j] = _fake(name, shapes, j, -1)
            assert call(a) == binding.LSTM_ERR_INVALID_ARG, (i, j)
    assert not lib.ran_on


@pytest.mark.parametrize("name", list(CALLS))
def test_addresses_alone(name, lib):
    call, shapes = CALLS[name]
    assert call([256] * len(shapes)) == binding.LSTM_OK
    assert lib.ran_on.pop() == 0

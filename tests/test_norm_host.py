"""lstm_layer_norm_*: sizes and what they refuse, before anything is enqueued (CPU)."""
import ctypes

import pytest
import torch

from layer_lstm_b200 import binding
from test_header_binding import C_SIZES, _header, _struct_fields

BIG = 1 << 40


def _fwd(desc, x=256, w=256, b=256, y=256, mean=256, rstd=256):
    return binding.lstm_layer_norm_forward(desc, x, w, b, y, mean, rstd, stream=0)


def _bwd(desc, gy=256, x=256, w=256, mean=256, rstd=256, dx=256, dw=256, db=256, ws=256, n=BIG):
    return binding.lstm_layer_norm_backward(desc, gy, x, w, mean, rstd, dx, dw, db, ws, stream=0, ws_bytes=n)


def test_struct_matches_header():
    fields = _struct_fields(_header(), "lstm_norm_desc")
    assert [n for _, n, _ in fields] == [n for n, _ in binding.lstm_norm_desc._fields_]
    for (typ, name, _), (_, ptype) in zip(fields, binding.lstm_norm_desc._fields_):
        assert ctypes.sizeof(ptype) == C_SIZES[typ], name


@pytest.mark.parametrize("kw", [dict(rows=-1), dict(cols=0), dict(dtype=2), dict(eps=-1e-5),
                                dict(eps=float("nan"))])
def test_refused_descriptions(kw):
    args = dict(rows=4, cols=8)
    args.update(kw)
    d = binding.make_norm_desc(**args)
    assert binding.lstm_layer_norm_workspace_size(d) == 0
    assert _fwd(d) == binding.LSTM_ERR_INVALID_ARG
    assert _bwd(d) == binding.LSTM_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(x=None), dict(y=None), dict(x=258), dict(y=257), dict(w=258), dict(b=258),
                                dict(mean=258), dict(rstd=258)])
def test_refused_forward_pointers(kw):
    assert _fwd(binding.make_norm_desc(4, 8), **kw) == binding.LSTM_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(gy=None), dict(x=None), dict(mean=None), dict(rstd=None), dict(dx=258),
                                dict(dw=258), dict(db=258), dict(ws=None), dict(ws=264), dict(gy=258)])
def test_refused_backward_pointers(kw):
    assert _bwd(binding.make_norm_desc(4, 8), **kw) == binding.LSTM_ERR_INVALID_ARG


def test_workspace():
    d = binding.make_norm_desc(1000, 100)
    need = binding.lstm_layer_norm_workspace_size(d)
    assert need > 0 and need % 256 == 0
    assert _bwd(d, n=need - 1) == binding.LSTM_ERR_WORKSPACE
    assert binding.lstm_layer_norm_workspace_size(binding.make_norm_desc(0, 100)) > 0


def test_nothing_to_do():
    d = binding.make_norm_desc(0, 8)
    assert _fwd(d, x=None, y=None) == binding.LSTM_OK
    assert _bwd(binding.make_norm_desc(4, 8), dx=None, dw=None, db=None, ws=None, n=0) == binding.LSTM_OK


def test_refused_tensors():
    d = binding.make_norm_desc(4, 8)
    x, v, s = torch.zeros(4, 8), torch.zeros(8), torch.zeros(4)
    # on the CPU, wrong type, wrong size, not contiguous
    for kw in (dict(x=x, y=x), dict(x=x.bfloat16()), dict(x=torch.zeros(4, 7)), dict(x=torch.zeros(8, 4).t()),
               dict(w=v.bfloat16()), dict(b=v[:7]), dict(mean=s.double()), dict(rstd=s[:3])):
        assert _fwd(d, **kw) == binding.LSTM_ERR_INVALID_ARG
    for kw in (dict(gy=x), dict(dw=v.bfloat16()), dict(db=v[:7]), dict(dx=x.double())):
        assert _bwd(d, **kw) == binding.LSTM_ERR_INVALID_ARG

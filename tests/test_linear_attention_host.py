"""lstm_linear_attention_*: sizes and what they refuse, before anything is enqueued (CPU)."""
import ctypes

import pytest
import torch

from layer_lstm_b200 import binding
from test_header_binding import C_SIZES, _header, _struct_fields

BIG = 1 << 40


def _fwd(d, lengths=None, q=256, k=256, v=256, ld=256, s0=256, out=256, s_n=256, ws=256, n=BIG):
    return binding.lstm_linear_attention_forward(d, q, k, v, ld, s0, out, s_n, ws, stream=0, ws_bytes=n,
                                                 lengths=lengths)


def _bwd(d, lengths=None, q=256, k=256, v=256, ld=256, s0=256, go=256, gs=256, dq=256, dk=256, dv=256, ds0=256,
         ws=256, n=BIG):
    return binding.lstm_linear_attention_backward(d, q, k, v, ld, s0, go, gs, dq, dk, dv, ds0, ws, stream=0,
                                                  ws_bytes=n, lengths=lengths)


def _step(d, lengths=None, q=256, k=256, v=256, ld=256, state=256, out=256):
    return binding.lstm_linear_attention_step(d, q, k, v, ld, state, out, stream=0, lengths=lengths)


def test_struct_matches_header():
    fields = _struct_fields(_header(), "lstm_attention_desc")
    assert [n for _, n, _ in fields] == [n for n, _ in binding.lstm_attention_desc._fields_]
    for (typ, name, _), (_, ptype) in zip(fields, binding.lstm_attention_desc._fields_):
        assert ctypes.sizeof(ptype) == C_SIZES[typ], name


@pytest.mark.parametrize("kw", [dict(batch=-1), dict(seq_len=-1), dict(heads=0), dict(key_size=0),
                                dict(value_size=0), dict(dtype=5), dict(scale=float("inf")),
                                dict(scale=float("nan")), dict(ld_q=15), dict(ld_k=1), dict(ld_v=-1)])
def test_refused_descriptions(kw):
    args = dict(batch=2, seq_len=1, heads=2, key_size=8, value_size=8)
    args.update(kw)
    d = binding.make_attention_desc(**args)
    assert binding.lstm_linear_attention_workspace_size(d) == 0
    for call in (_fwd, _bwd, _step):
        assert call(d) == binding.LSTM_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(key_size=129), dict(value_size=200), dict(seq_len=(1 << 30) + 1)])
def test_unsupported_sizes(kw):
    args = dict(batch=2, seq_len=1, heads=2, key_size=8, value_size=8)
    args.update(kw)
    d = binding.make_attention_desc(**args)
    assert binding.lstm_linear_attention_workspace_size(d) == 0
    for call in (_fwd, _bwd) + ((_step,) if "seq_len" not in kw else ()):
        assert call(d) == binding.LSTM_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw", [dict(q=None), dict(k=None), dict(v=None), dict(ld=None), dict(out=None), dict(ws=None),
                                dict(q=258), dict(k=257), dict(v=258), dict(out=258), dict(ld=258), dict(s0=258),
                                dict(s_n=258), dict(ws=264), dict(lengths=258)])
def test_refused_forward_pointers(kw):
    assert _fwd(binding.make_attention_desc(2, 3, 2, 8, 8), **kw) == binding.LSTM_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(q=None), dict(k=None), dict(v=None), dict(ld=None), dict(go=None), dict(dq=None),
                                dict(dk=None), dict(dv=None), dict(ws=None), dict(go=258), dict(gs=258),
                                dict(ds0=258), dict(lengths=257), dict(dv=258)])
def test_refused_backward_pointers(kw):
    assert _bwd(binding.make_attention_desc(2, 3, 2, 8, 8), **kw) == binding.LSTM_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(q=None), dict(k=None), dict(v=None), dict(ld=None), dict(state=None),
                                dict(out=None), dict(state=258), dict(out=257), dict(lengths=258)])
def test_refused_step_pointers(kw):
    assert _step(binding.make_attention_desc(2, 1, 2, 8, 8), **kw) == binding.LSTM_ERR_INVALID_ARG


def test_step_takes_one_token():
    assert _step(binding.make_attention_desc(2, 2, 2, 8, 8)) == binding.LSTM_ERR_INVALID_ARG


def test_workspace():
    small = binding.lstm_linear_attention_workspace_size(binding.make_attention_desc(64, 128, 8, 64, 64))
    d = binding.make_attention_desc(1, 32768, 2, 128, 128)
    need = binding.lstm_linear_attention_workspace_size(d)
    assert 0 < small < need and need % 256 == 0
    assert _fwd(d, n=need - 1) == binding.LSTM_ERR_WORKSPACE
    assert _bwd(d, n=need - 1) == binding.LSTM_ERR_WORKSPACE


def test_empty_batch():
    d = binding.make_attention_desc(0, 3, 2, 8, 8)
    assert _fwd(d, q=None, k=None, v=None, out=None) == binding.LSTM_OK
    assert _bwd(d, q=None, k=None, v=None, go=None, dq=None, dk=None, dv=None) == binding.LSTM_OK
    assert _step(binding.make_attention_desc(0, 1, 2, 8, 8), q=None, state=None, out=None) == binding.LSTM_OK


def test_refused_tensors():
    d = binding.make_attention_desc(2, 3, 2, 8, 8)
    x, ld, s = torch.zeros(2, 3, 2, 8), torch.zeros(2), torch.zeros(2, 2, 8, 8)
    wide = torch.zeros(2, 3, 3, 2, 8)
    for kw in (dict(q=x), dict(q=x.bfloat16()), dict(k=x[:, :2]), dict(v=wide[:, :, 1]), dict(out=wide[:, :, 0]),
               dict(ld=ld.double()), dict(s0=s.bfloat16()), dict(s_n=s[:1]), dict(q=x.transpose(0, 1)),
               dict(lengths=torch.zeros(2, dtype=torch.int64))):
        assert _fwd(d, **kw) == binding.LSTM_ERR_INVALID_ARG
    for kw in (dict(dq=x.bfloat16()), dict(go=x[:1]), dict(gs=s.double()), dict(ds0=s[0])):
        assert _bwd(d, **kw) == binding.LSTM_ERR_INVALID_ARG


def test_packed_rows_are_recognised():
    B, T, H, dk, dv = 2, 3, 2, 8, 4
    row = 2 * H * dk + H * dv
    d = binding.make_attention_desc(B, T, H, dk, dv, ld_q=row, ld_k=row, ld_v=row)
    p = torch.zeros(B, T, row)
    q = p[..., :H * dk].view(B, T, H, dk)
    k = p[..., H * dk:2 * H * dk].view(B, T, H, dk)
    v = p[..., 2 * H * dk:].view(B, T, H, dv)
    cpu = -1   # a CPU tensor's device index
    for t, size, ld in ((q, dk, d.ld_q), (k, dk, d.ld_k), (v, dv, d.ld_v)):
        assert binding._fits_rows(t, d, size, ld, torch.float32, cpu)
        assert not binding._fits_rows(t, d, size, 0, torch.float32, cpu)
        assert not binding._fits_rows(t.contiguous(), d, size, ld, torch.float32, cpu)

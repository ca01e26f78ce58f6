"""Thin ctypes binding of liblstm_b200.so (include/lstm.h).

Argument marshalling only: tensors become device pointers, lists of tensors
become host arrays of device pointers, and every function returns the C
status code.  All computation happens in the CUDA library; there is no other
code path.  PyTorch is used by callers for device memory and streams; calls
with plain addresses and a stream handle do without it.
"""
from __future__ import annotations

import ctypes
import os

from . import build as _build

LSTM_OK = 0
LSTM_ERR_INVALID_ARG = 1
LSTM_ERR_UNSUPPORTED = 2
LSTM_ERR_WORKSPACE = 3
LSTM_ERR_CUDA = 4
LSTM_ERR_TIMEOUT = 5
LSTM_F32 = 0
LSTM_BF16 = 1

EXPORTED = ("lstm_workspace_size", "lstm_reserve_size", "lstm_forward", "lstm_backward",
            "lstm_query_status", "lstm_status_string", "lstm_timing_enable", "lstm_timing_read",
            "lstm_timing_reset", "lstm_forward_noalloc", "lstm_trace_enable", "lstm_trace_read",
            "lstm_forward_varlen", "lstm_backward_varlen", "lstm_noalloc_query_status", "lstm_adamw_step",
            "lstm_adamw_read_state", "lstm_layer_norm_workspace_size", "lstm_layer_norm_forward",
            "lstm_layer_norm_backward", "lstm_linear_attention_workspace_size", "lstm_linear_attention_forward",
            "lstm_linear_attention_backward", "lstm_linear_attention_step")
LSTM_NOALLOC_SCRATCH_BYTES = 32 << 20
LSTM_TRACE_MAX_STEPS = 512
LSTM_TRACE_EVENTS = 16
LSTM_TRACE_FWD_REC_FFMA = 1
LSTM_TRACE_BWD_REC_FFMA = 2
LSTM_TRACE_FWD_REC_TC = 3
LSTM_TRACE_FWD_REC_TC32 = 4
LSTM_TRACE_BWD_REC_TC32 = 5


class lstm_kernel_time(ctypes.Structure):
    _fields_ = [("name", ctypes.c_char_p), ("launches", ctypes.c_longlong),
                ("total_ms", ctypes.c_double)]


class lstm_desc(ctypes.Structure):
    _fields_ = [("input_size", ctypes.c_int), ("hidden_size", ctypes.c_int),
                ("num_layers", ctypes.c_int), ("bidirectional", ctypes.c_int),
                ("bias", ctypes.c_int), ("batch_first", ctypes.c_int),
                ("batch", ctypes.c_int), ("seq_len", ctypes.c_int), ("dtype", ctypes.c_int),
                ("dropout", ctypes.c_float), ("dropout_seed", ctypes.c_ulonglong)]


class lstm_adamw_desc(ctypes.Structure):
    _fields_ = [("num_tensors", ctypes.c_int), ("grad_dtype", ctypes.c_int), ("state_bits", ctypes.c_int),
                ("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("weight_decay", ctypes.c_double), ("seed", ctypes.c_ulonglong)]


class lstm_norm_desc(ctypes.Structure):
    _fields_ = [("rows", ctypes.c_longlong), ("cols", ctypes.c_int), ("dtype", ctypes.c_int),
                ("eps", ctypes.c_float)]


class lstm_attention_desc(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int), ("seq_len", ctypes.c_int), ("heads", ctypes.c_int),
                ("key_size", ctypes.c_int), ("value_size", ctypes.c_int), ("batch_first", ctypes.c_int),
                ("dtype", ctypes.c_int), ("scale", ctypes.c_float), ("ld_q", ctypes.c_longlong),
                ("ld_k", ctypes.c_longlong), ("ld_v", ctypes.c_longlong)]


def make_desc(input_size, hidden_size, num_layers=1, bidirectional=False, bias=True,
              batch_first=True, batch=1, seq_len=1, dtype=LSTM_F32, dropout=0.0,
              dropout_seed=0) -> lstm_desc:
    return lstm_desc(int(input_size), int(hidden_size), int(num_layers), int(bool(bidirectional)),
                     int(bool(bias)), int(bool(batch_first)), int(batch), int(seq_len), int(dtype),
                     float(dropout), int(dropout_seed))


def make_adamw_desc(num_tensors, grad_dtype=LSTM_F32, state_bits=32, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8,
                    weight_decay=0.01, seed=0) -> lstm_adamw_desc:
    return lstm_adamw_desc(int(num_tensors), int(grad_dtype), int(state_bits), float(lr), float(beta1),
                           float(beta2), float(eps), float(weight_decay), int(seed))


def make_norm_desc(rows, cols, dtype=LSTM_F32, eps=1e-5) -> lstm_norm_desc:
    return lstm_norm_desc(int(rows), int(cols), int(dtype), float(eps))


def make_attention_desc(batch, seq_len, heads, key_size, value_size, batch_first=True, dtype=LSTM_F32, scale=None,
                        ld_q=0, ld_k=0, ld_v=0) -> lstm_attention_desc:
    """scale: None for key_size ** -0.5; ld_*: elements between time rows, 0 for rows without a gap."""
    return lstm_attention_desc(int(batch), int(seq_len), int(heads), int(key_size), int(value_size),
                               int(bool(batch_first)), int(dtype),
                               float(max(key_size, 1) ** -0.5 if scale is None else scale), int(ld_q), int(ld_k),
                               int(ld_v))


_lib = None


class LstmError(RuntimeError):
    def __init__(self, status, where=""):
        super().__init__(f"{where}: {status_string(status)} ({status})")
        self.status = status


def lib_path() -> str:
    return _build.LIB_PATH


def load(build_if_stale: bool = True):
    """Loads the CUDA library (building it in-tree when sources are newer).

    Raises if the library cannot be built or loaded: there is no fallback."""
    global _lib
    if _lib is not None:
        return _lib
    if build_if_stale:
        _build.build()
    if not os.path.exists(_build.LIB_PATH):
        raise RuntimeError(f"CUDA library missing: {_build.LIB_PATH}")
    lib = ctypes.CDLL(_build.LIB_PATH)
    vp = ctypes.c_void_p
    vpp = ctypes.POINTER(ctypes.c_void_p)
    dp = ctypes.POINTER(lstm_desc)
    sz = ctypes.c_size_t
    lib.lstm_workspace_size.argtypes = [dp]
    lib.lstm_workspace_size.restype = sz
    lib.lstm_reserve_size.argtypes = [dp]
    lib.lstm_reserve_size.restype = sz
    lib.lstm_forward.argtypes = [dp, vp, vp, vp, vpp, vpp, vpp, vpp, vp, vp, vp, vp, sz, vp, sz, vp]
    lib.lstm_forward.restype = ctypes.c_int
    lib.lstm_backward.argtypes = [dp, vp, vp, vp, vpp, vpp, vp, vp, vp, vp, sz, vp, sz, vp, vp, vp,
                                  vpp, vpp, vpp, vpp, vp]
    lib.lstm_backward.restype = ctypes.c_int
    lib.lstm_forward_varlen.argtypes = [dp, vp] + list(lib.lstm_forward.argtypes[1:])
    lib.lstm_forward_varlen.restype = ctypes.c_int
    lib.lstm_backward_varlen.argtypes = [dp, vp] + list(lib.lstm_backward.argtypes[1:])
    lib.lstm_backward_varlen.restype = ctypes.c_int
    lib.lstm_query_status.argtypes = [vp, vp]
    lib.lstm_query_status.restype = ctypes.c_int
    lib.lstm_status_string.argtypes = [ctypes.c_int]
    lib.lstm_status_string.restype = ctypes.c_char_p
    lib.lstm_timing_enable.argtypes = [ctypes.c_int]
    lib.lstm_timing_enable.restype = ctypes.c_int
    lib.lstm_timing_read.argtypes = [ctypes.POINTER(lstm_kernel_time), ctypes.c_int]
    lib.lstm_timing_read.restype = ctypes.c_int
    lib.lstm_timing_reset.argtypes = []
    lib.lstm_timing_reset.restype = None
    lib.lstm_forward_noalloc.argtypes = [dp, vp, vp, vp, vpp, vpp, vpp, vpp, vp, vp, vp, vp]
    lib.lstm_forward_noalloc.restype = ctypes.c_int
    lib.lstm_noalloc_query_status.argtypes = [vp]
    lib.lstm_noalloc_query_status.restype = ctypes.c_int
    lib.lstm_trace_enable.argtypes = [ctypes.c_int]
    lib.lstm_trace_enable.restype = ctypes.c_int
    lib.lstm_trace_read.argtypes = [ctypes.POINTER(ctypes.c_ulonglong), ctypes.c_int, ctypes.POINTER(ctypes.c_int)]
    lib.lstm_trace_read.restype = ctypes.c_int
    ap = ctypes.POINTER(lstm_adamw_desc)
    lp = ctypes.POINTER(ctypes.c_longlong)
    lib.lstm_adamw_step.argtypes = [ap, lp] + [vpp] * 7 + [vp, vp, vp]
    lib.lstm_adamw_step.restype = ctypes.c_int
    lib.lstm_adamw_read_state.argtypes = [ap, lp] + [vpp] * 6 + [vp]
    lib.lstm_adamw_read_state.restype = ctypes.c_int
    np_ = ctypes.POINTER(lstm_norm_desc)
    lib.lstm_layer_norm_workspace_size.argtypes = [np_]
    lib.lstm_layer_norm_workspace_size.restype = sz
    lib.lstm_layer_norm_forward.argtypes = [np_] + [vp] * 7
    lib.lstm_layer_norm_forward.restype = ctypes.c_int
    lib.lstm_layer_norm_backward.argtypes = [np_] + [vp] * 9 + [sz, vp]
    lib.lstm_layer_norm_backward.restype = ctypes.c_int
    tp = ctypes.POINTER(lstm_attention_desc)
    lib.lstm_linear_attention_workspace_size.argtypes = [tp]
    lib.lstm_linear_attention_workspace_size.restype = sz
    lib.lstm_linear_attention_forward.argtypes = [tp] + [vp] * 9 + [sz, vp]
    lib.lstm_linear_attention_forward.restype = ctypes.c_int
    lib.lstm_linear_attention_backward.argtypes = [tp] + [vp] * 13 + [sz, vp]
    lib.lstm_linear_attention_backward.restype = ctypes.c_int
    lib.lstm_linear_attention_step.argtypes = [tp] + [vp] * 8
    lib.lstm_linear_attention_step.restype = ctypes.c_int
    _lib = lib
    return lib


def _p(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _nbytes(t):
    if t is None:
        return 0
    return t.numel() * t.element_size()


def _parr(ts):
    if ts is None:
        return None
    return (ctypes.c_void_p * len(ts))(*[_p(t) for t in ts])


def _stream(stream):
    if stream is None:
        import torch
        # the handle alone: torch.cuda.current_stream() builds an object around it (3.4 us of a 13 us call)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def status_string(status: int) -> str:
    return load().lstm_status_string(int(status)).decode()


def lstm_status_string(status: int) -> str:
    return status_string(status)


def lstm_workspace_size(desc: lstm_desc) -> int:
    return int(load().lstm_workspace_size(ctypes.byref(desc)))


def lstm_reserve_size(desc: lstm_desc) -> int:
    return int(load().lstm_reserve_size(ctypes.byref(desc)))


def lstm_forward(desc, x, h0, c0, w_ih, w_hh, b_ih, b_hh, out, h_n, c_n, workspace,
                 reserve=None, stream=None, ws_bytes=None, rs_bytes=None, lengths=None) -> int:
    """lengths: device int32 tensor of per-row valid steps (lstm_forward_varlen),
    or None (lstm_forward)."""
    lib = load()
    args = (_p(x), _p(h0), _p(c0), _parr(w_ih), _parr(w_hh),
            _parr(b_ih), _parr(b_hh), _p(out), _p(h_n), _p(c_n),
            _p(workspace), _nbytes(workspace) if ws_bytes is None else ws_bytes,
            _p(reserve), _nbytes(reserve) if rs_bytes is None else rs_bytes,
            _stream(stream))
    if lengths is None:
        return lib.lstm_forward(ctypes.byref(desc), *args)
    return lib.lstm_forward_varlen(ctypes.byref(desc), _p(lengths), *args)


def lstm_backward(desc, x, h0, c0, w_ih, w_hh, grad_out, grad_hn, grad_cn, reserve, workspace,
                  dx, dh0, dc0, dw_ih, dw_hh, db_ih, db_hh, stream=None,
                  ws_bytes=None, rs_bytes=None, lengths=None) -> int:
    lib = load()
    args = (_p(x), _p(h0), _p(c0), _parr(w_ih), _parr(w_hh),
            _p(grad_out), _p(grad_hn), _p(grad_cn), _p(reserve),
            _nbytes(reserve) if rs_bytes is None else rs_bytes,
            _p(workspace), _nbytes(workspace) if ws_bytes is None else ws_bytes,
            _p(dx), _p(dh0), _p(dc0), _parr(dw_ih), _parr(dw_hh),
            _parr(db_ih), _parr(db_hh), _stream(stream))
    if lengths is None:
        return lib.lstm_backward(ctypes.byref(desc), *args)
    return lib.lstm_backward_varlen(ctypes.byref(desc), _p(lengths), *args)


def lstm_forward_noalloc(desc, x, h0, c0, w_ih, w_hh, b_ih, b_hh, out, h_n, c_n,
                         stream=None) -> int:
    lib = load()
    return lib.lstm_forward_noalloc(ctypes.byref(desc), _p(x), _p(h0), _p(c0), _parr(w_ih),
                                    _parr(w_hh), _parr(b_ih), _parr(b_hh), _p(out), _p(h_n),
                                    _p(c_n), _stream(stream))


def lstm_noalloc_query_status(stream=None) -> int:
    return int(load().lstm_noalloc_query_status(_stream(stream)))


def lstm_query_status(workspace, stream=None) -> int:
    return int(load().lstm_query_status(_p(workspace), _stream(stream)))


def lstm_timing_enable(enable: bool) -> int:
    return int(load().lstm_timing_enable(int(bool(enable))))


def lstm_timing_reset() -> None:
    load().lstm_timing_reset()


def lstm_timing_read() -> dict:
    """{kind: (launches, total_ms)} accumulated since the last reset."""
    lib = load()
    n = lib.lstm_timing_read(None, 0)
    arr = (lstm_kernel_time * n)()
    got = lib.lstm_timing_read(arr, n)
    if got < 0:
        raise LstmError(LSTM_ERR_CUDA, "lstm_timing_read")
    return {arr[i].name.decode(): (int(arr[i].launches), float(arr[i].total_ms)) for i in range(got)}


def lstm_trace_enable(enable: bool) -> int:
    return int(load().lstm_trace_enable(int(bool(enable))))


def lstm_trace_read(max_steps: int = LSTM_TRACE_MAX_STEPS):
    """(kind, rows): rows is a list of LSTM_TRACE_EVENTS-long lists of
    %globaltimer stamps (ns) of the last traced recurrent launch."""
    lib = load()
    buf = (ctypes.c_ulonglong * (max_steps * LSTM_TRACE_EVENTS))()
    kind = ctypes.c_int(0)
    n = lib.lstm_trace_read(buf, max_steps, ctypes.byref(kind))
    if n < 0:
        raise LstmError(LSTM_ERR_CUDA, "lstm_trace_read")
    rows = [list(buf[i * LSTM_TRACE_EVENTS:(i + 1) * LSTM_TRACE_EVENTS]) for i in range(n)]
    return int(kind.value), rows


def _numels(ts):
    return (ctypes.c_longlong * len(ts))(*[int(t) for t in ts])


def lstm_adamw_step(desc, numel, param, param_bf16, grad, m, v, m_scale, v_scale, step, scalars=None,
                    stream=None) -> int:
    """numel: ints; the other lists: tensors, device addresses or None entries (see optim.AdamW, which
    keeps these arrays and checks the tensors).  Lists already made into ctypes arrays pass as they are."""
    a = [x if x is None or isinstance(x, ctypes.Array) else _parr(x)
         for x in (param, param_bf16, grad, m, v, m_scale, v_scale)]
    n = numel if isinstance(numel, ctypes.Array) else _numels(numel)
    return load().lstm_adamw_step(ctypes.byref(desc), n, *a, _p(step), _p(scalars), _stream(stream))


def lstm_adamw_read_state(desc, numel, m, v, m_scale, v_scale, m_out, v_out, stream=None) -> int:
    a = [x if x is None or isinstance(x, ctypes.Array) else _parr(x)
         for x in (m, v, m_scale, v_scale, m_out, v_out)]
    n = numel if isinstance(numel, ctypes.Array) else _numels(numel)
    return load().lstm_adamw_read_state(ctypes.byref(desc), n, *a, _stream(stream))


_TYPES = {}   # torch's types by name or code, known once a call brings a tensor


def _fits(t, numel, dtype, device):
    """Whether `t` is what a call reads as `numel` contiguous elements of `dtype` on GPU `device`: a tensor
    of that kind, a plain device address, or None (an argument left out)."""
    if t is None or isinstance(t, int):
        return True
    return t.dtype is dtype and t.numel() == numel and t.get_device() == device and t.is_contiguous()


def _device(*ts):
    """Index of the GPU of the first tensor among a call's arguments (-1: a CPU tensor); None when all are
    plain addresses."""
    for t in ts:
        if t is not None and not isinstance(t, int):
            if not _TYPES:
                import torch
                _TYPES.update({LSTM_F32: torch.float32, LSTM_BF16: torch.bfloat16, "f32": torch.float32,
                               "i32": torch.int32})
            return t.get_device()
    return None


def _call(device, stream, f, *args):
    """f(*args, stream handle) with GPU `device` current, so that a call on another device's tensors runs
    there, on `stream` or that device's current stream.  Tensors that are not on a GPU are refused."""
    if device is not None and device < 0:
        return LSTM_ERR_INVALID_ARG
    if device is None:
        return f(*args, _stream(stream))
    import torch
    if device == torch.cuda.current_device():
        return f(*args, _stream(stream))
    with torch.cuda.device(device):
        return f(*args, _stream(stream))


def lstm_layer_norm_workspace_size(desc: lstm_norm_desc) -> int:
    return int(load().lstm_layer_norm_workspace_size(ctypes.byref(desc)))


def lstm_layer_norm_forward(desc, x, weight, bias, y, mean=None, rstd=None, stream=None) -> int:
    """Tensors whose type, device, size or contiguity does not match the description are refused
    (LSTM_ERR_INVALID_ARG); plain device addresses pass as they are."""
    rows, cols, dev = desc.rows, desc.cols, _device(x, y, weight, bias, mean, rstd)
    dt, f32 = _TYPES.get(desc.dtype), _TYPES.get("f32")
    if not (_fits(x, rows * cols, dt, dev) and _fits(y, rows * cols, dt, dev) and _fits(weight, cols, dt, dev)
            and _fits(bias, cols, dt, dev) and _fits(mean, rows, f32, dev) and _fits(rstd, rows, f32, dev)):
        return LSTM_ERR_INVALID_ARG
    return _call(dev, stream, load().lstm_layer_norm_forward, ctypes.byref(desc), _p(x), _p(weight), _p(bias), _p(y),
                 _p(mean), _p(rstd))


def lstm_layer_norm_backward(desc, grad_y, x, weight, mean, rstd, dx, dweight, dbias, workspace=None, stream=None,
                             ws_bytes=None) -> int:
    rows, cols, dev = desc.rows, desc.cols, _device(grad_y, x, weight, mean, rstd, dx, dweight, dbias, workspace)
    n, dt, f32 = rows * cols, _TYPES.get(desc.dtype), _TYPES.get("f32")
    if not (_fits(grad_y, n, dt, dev) and _fits(x, n, dt, dev) and _fits(dx, n, dt, dev)
            and _fits(weight, cols, dt, dev) and _fits(mean, rows, f32, dev) and _fits(rstd, rows, f32, dev)
            and _fits(dweight, cols, f32, dev) and _fits(dbias, cols, f32, dev)
            and _device(workspace) in (None, dev)):
        return LSTM_ERR_INVALID_ARG
    return _call(dev, stream, load().lstm_layer_norm_backward, ctypes.byref(desc), _p(grad_y), _p(x), _p(weight),
                 _p(mean), _p(rstd), _p(dx), _p(dweight), _p(dbias), _p(workspace),
                 _nbytes(workspace) if ws_bytes is None else ws_bytes)


def lstm_linear_attention_workspace_size(desc: lstm_attention_desc) -> int:
    return int(load().lstm_linear_attention_workspace_size(ctypes.byref(desc)))


def _fits_rows(t, desc, size, ld, dtype, device):
    """Whether `t` is an array of desc's time rows, heads and `size` elements, the rows `ld` apart (0: no
    gap): an address, a tensor of four dimensions, or a contiguous one of another shape."""
    if t is None or isinstance(t, int):
        return True
    n, row = t.numel(), desc.heads * size
    if t.dtype is not dtype or t.get_device() != device or n != desc.batch * desc.seq_len * row:
        return False
    ld = ld or row
    if n == 0 or (ld == row and t.is_contiguous()):
        return True
    if t.dim() != 4 or t.shape[2] != desc.heads or t.shape[3] != size:
        return False
    outer, inner, s = t.shape[0], t.shape[1], t.stride()
    if (outer, inner) != ((desc.batch, desc.seq_len) if desc.batch_first else (desc.seq_len, desc.batch)):
        return False
    return ((size == 1 or s[3] == 1) and (desc.heads == 1 or s[2] == size) and (inner == 1 or s[1] == ld)
            and (outer == 1 or s[0] == inner * ld))


def _attention_fits(desc, dev, lengths, log_decay, qs, ks, vs, outs, states, workspace=None):
    dt, f32 = _TYPES.get(desc.dtype), _TYPES.get("f32")
    dk, dv = desc.key_size, desc.value_size
    n = desc.batch * desc.heads * dk * dv
    for ts, size, ld in ((qs, dk, desc.ld_q), (ks, dk, desc.ld_k), (vs, dv, desc.ld_v), (outs, dv, 0)):
        for t in ts:
            if not _fits_rows(t, desc, size, ld, dt, dev):
                return False
    for t in states:
        if not _fits(t, n, f32, dev):
            return False
    return (_fits(log_decay, desc.heads, f32, dev) and _fits(lengths, desc.batch, _TYPES.get("i32"), dev)
            and _device(workspace) in (None, dev))


def lstm_linear_attention_forward(desc, q, k, v, log_decay, s0, out, s_n, workspace, stream=None, ws_bytes=None,
                                  lengths=None) -> int:
    """Tensors that do not match the description (type, device, size, layout) are refused with
    LSTM_ERR_INVALID_ARG; plain device addresses pass as they are."""
    dev = _device(q, k, v, log_decay, s0, out, s_n, workspace, lengths)
    if not _attention_fits(desc, dev, lengths, log_decay, (q,), (k,), (v,), (out,), (s0, s_n), workspace):
        return LSTM_ERR_INVALID_ARG
    return _call(dev, stream, load().lstm_linear_attention_forward, ctypes.byref(desc), _p(lengths), _p(q), _p(k),
                 _p(v), _p(log_decay), _p(s0), _p(out), _p(s_n), _p(workspace),
                 _nbytes(workspace) if ws_bytes is None else ws_bytes)


def lstm_linear_attention_backward(desc, q, k, v, log_decay, s0, grad_out, grad_sn, dq, dk, dv, ds0, workspace,
                                   stream=None, ws_bytes=None, lengths=None) -> int:
    dev = _device(q, k, v, log_decay, s0, grad_out, grad_sn, dq, dk, dv, ds0, workspace, lengths)
    if not _attention_fits(desc, dev, lengths, log_decay, (q, dq), (k, dk), (v, dv), (grad_out,),
                           (s0, grad_sn, ds0), workspace):
        return LSTM_ERR_INVALID_ARG
    return _call(dev, stream, load().lstm_linear_attention_backward, ctypes.byref(desc), _p(lengths), _p(q), _p(k),
                 _p(v), _p(log_decay), _p(s0), _p(grad_out), _p(grad_sn), _p(dq), _p(dk), _p(dv), _p(ds0),
                 _p(workspace), _nbytes(workspace) if ws_bytes is None else ws_bytes)


def lstm_linear_attention_step(desc, q, k, v, log_decay, state, out, stream=None, lengths=None) -> int:
    dev = _device(q, k, v, log_decay, state, out, lengths)
    if not _attention_fits(desc, dev, lengths, log_decay, (q,), (k,), (v,), (out,), (state,)):
        return LSTM_ERR_INVALID_ARG
    return _call(dev, stream, load().lstm_linear_attention_step, ctypes.byref(desc), _p(lengths), _p(q), _p(k), _p(v),
                 _p(log_decay), _p(state), _p(out))


def check(status: int, where: str = "lstm") -> None:
    if status != LSTM_OK:
        raise LstmError(status, where)

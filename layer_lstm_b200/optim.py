"""AdamW over the tensors of a model, on the library's multi-tensor kernel.

`AdamW` holds the moments and the step counter on the GPU and keeps the
pointer arrays that lstm_adamw_step takes for as long as the tensors are the
same, so a step costs one call.  The
gradients are read from the tensors it was given (for a training problem:
the gradient tensors the LSTM backward overwrites, or the views of a
dp.GradBucket), the parameters are updated in place and, where the layers
compute in bf16, written to their bf16 tensors too.
"""
from __future__ import annotations

import bisect
import ctypes

import torch

from . import binding

BLOCK = 256   # elements of a tensor that share one scale of the 8-bit moments


def _check(name, t, dtype, device, numel):
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or t.device != device or t.numel() != numel \
            or not t.is_contiguous():
        raise ValueError(f"{name}: need a contiguous {dtype} tensor of {numel} elements on {device}")


def _spans(ts):
    return [(at, at + n) for at, n in ((t.data_ptr(), t.nbytes) for t in ts) if n]


def _check_apart(written, read):
    """The tensors of `written` share no memory with one another or with those of `read`."""
    spans = sorted(_spans(written))
    for (_, end), (start, _) in zip(spans, spans[1:]):
        if start < end:
            raise ValueError("parameters, copies and moments may not share memory")
    for start, end in _spans(read):
        i = bisect.bisect_left(spans, (end,))   # the spans that begin before its end
        if i and spans[i - 1][1] > start:
            raise ValueError("a gradient may not share memory with what a step writes")


class AdamW:
    """params: float32 tensors; grads: as many float32 or bf16 tensors (one type) of the same sizes.  What a
    step writes may not share memory (a weight used twice is given once).

    copies: bf16 tensors (or None entries) that receive the updated parameters.  state_bits: 32, or 8
    (codes in blocks of 256 elements; see include/lstm.h).  scalars: float32 device tensor of two, the
    factors of the learning rate and of the gradients, read at every step (a schedule or a loss scale
    that a captured graph follows).  state: moments and step counter of an earlier run, a dict as
    `state` of this class; they are used in place, not copied.

    A step takes the tensors that params, grads, copies and state hold when it is called: entries may be
    replaced between steps by others of the same kind (checked then, ValueError).  A captured step keeps
    the tensors it was captured with, which the caller keeps alive."""

    def __init__(self, params, grads, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01,
                 copies=None, state_bits=32, seed=0, scalars=None, state=None):
        self.params, self.grads = list(params), list(grads)
        self.copies = list(copies) if copies is not None else None
        if state_bits not in (8, 32):
            raise ValueError("state_bits is 8 or 32")
        n = len(self.params)
        self.device = self.params[0].device if n else torch.device("cuda", torch.cuda.current_device())
        self.scalars = scalars
        self.desc = binding.make_adamw_desc(n, binding.LSTM_F32, state_bits, lr, beta1, beta2, eps, weight_decay,
                                            seed)
        if state is None:
            eight, device = state_bits == 8, self.device
            mdt, vdt = (torch.int8, torch.uint8) if eight else (torch.float32, torch.float32)
            state = dict(m=[torch.zeros(p.shape, device=device, dtype=mdt) for p in self.params],
                         v=[torch.zeros(p.shape, device=device, dtype=vdt) for p in self.params],
                         m_scale=None, v_scale=None, step=torch.zeros(1, device=device, dtype=torch.int64))
            if eight:
                for name in ("m_scale", "v_scale"):
                    state[name] = [torch.zeros(-(-p.numel() // BLOCK), device=device) for p in self.params]
        self.state = state
        self._take()

    def _lists(self):
        """The lists of tensors that lstm_adamw_step takes, in its order."""
        s, eight = self.state, self.desc.state_bits == 8
        return (self.params, self.copies, self.grads, s["m"], s["v"], s["m_scale"] if eight else None,
                s["v_scale"] if eight else None)

    def _addresses(self):
        a = []
        for ts in self._lists():
            if ts is self.copies:   # (entries may be None)
                a += [t is not None and t.data_ptr() for t in ts or ()]
            elif ts is not None:
                a += map(torch.Tensor.data_ptr, ts)
        a.append(self.state["step"].data_ptr())
        if self.scalars is not None:
            a.append(self.scalars.data_ptr())
        return a

    def _take(self):
        """Checks the tensors, holds them, and makes their pointer arrays."""
        n, device, eight, state = len(self.params), self.device, self.desc.state_bits == 8, self.state
        if len(self.grads) != n or (self.copies is not None and len(self.copies) != n):
            raise ValueError("one gradient (and one copy) for each parameter")
        gdt = self.grads[0].dtype if n else torch.float32
        if gdt not in (torch.float32, torch.bfloat16):
            raise ValueError("gradients are float32 or bf16")
        sizes = [p.numel() for p in self.params]
        for i, k in enumerate(sizes):
            _check(f"params[{i}]", self.params[i], torch.float32, device, k)
            _check(f"grads[{i}]", self.grads[i], gdt, device, k)
            if self.copies is not None and self.copies[i] is not None:
                _check(f"copies[{i}]", self.copies[i], torch.bfloat16, device, k)
        if self.scalars is not None:
            _check("scalars", self.scalars, torch.float32, device, 2)
        for name, dt, div in (("m", torch.int8 if eight else torch.float32, 1),
                              ("v", torch.uint8 if eight else torch.float32, 1),
                              ("m_scale", torch.float32, BLOCK), ("v_scale", torch.float32, BLOCK)):
            if div > 1 and not eight:
                continue
            if len(state[name]) != n:
                raise ValueError(f"state: one {name} for each parameter")
            for i, k in enumerate(sizes):
                _check(f"{name}[{i}]", state[name][i], dt, device, -(-k // div))
        _check("step", state["step"], torch.int64, device, 1)
        _check_apart([t for ts in self._lists() if ts is not None and ts is not self.grads for t in ts if t is not None]
                     + [state["step"]], self.grads)
        self.desc.num_tensors = n
        self.desc.grad_dtype = binding.LSTM_F32 if gdt == torch.float32 else binding.LSTM_BF16
        self._numel = binding._numels(sizes)
        self._at = [sum(sizes[:i]) for i in range(n)]   # where each tensor starts in the flat moments
        lists = self._lists()
        self._held = [list(ts) for ts in lists if ts is not None]   # what the arrays point to stays alive
        self._ptr = [binding._parr(ts) for ts in lists]
        self._taken = self._addresses()

    def _follow(self):
        """Takes the tensors anew where one was replaced, or its storage (a checkpoint restored into
        `state`, gradients moved into a bucket): the pointer arrays are of the tensors as they are now."""
        if self._addresses() != self._taken:
            self._take()

    def step(self, stream=None) -> None:
        """One update of every tensor, on `stream` (default: the current stream of the tensors' device)."""
        self._follow()
        p = self._ptr
        if self.device.index == torch.cuda.current_device():
            st = binding.lstm_adamw_step(self.desc, self._numel, *p, self.state["step"], self.scalars, stream)
        else:
            with torch.cuda.device(self.device):
                st = binding.lstm_adamw_step(self.desc, self._numel, *p, self.state["step"], self.scalars, stream)
        binding.check(st, "lstm_adamw_step")

    def read_state(self, m_out=None, v_out=None, stream=None):
        """The moments as two flat float32 tensors, every parameter's after the one before, written on
        `stream` (default: the current stream of the tensors' device; what is not given is that stream's)."""
        self._follow()
        total = sum(self._numel)
        with torch.cuda.device(self.device):
            s = torch.cuda.current_stream() if stream is None else stream
            s = torch.cuda.ExternalStream(s) if isinstance(s, int) else s
            with torch.cuda.stream(s):
                if m_out is None:
                    m_out = torch.empty(total, device=self.device)
                if v_out is None:
                    v_out = torch.empty(total, device=self.device)
                for name, t in (("m_out", m_out), ("v_out", v_out)):
                    _check(name, t, torch.float32, self.device, total)
                if self.desc.state_bits == 32:
                    for out, ts in ((m_out, self.state["m"]), (v_out, self.state["v"])):
                        if ts:
                            torch.cat([t.reshape(-1) for t in ts], out=out)
                    return m_out, v_out
                outs = [(ctypes.c_void_p * len(self.params))(*[t.data_ptr() + 4 * at for at in self._at])
                        for t in (m_out, v_out)]
                st = binding.lstm_adamw_read_state(self.desc, self._numel, *self._ptr[3:], *outs, s)
        binding.check(st, "lstm_adamw_read_state")
        return m_out, v_out

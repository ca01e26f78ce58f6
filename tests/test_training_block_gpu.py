"""The operators together, as a training step of a small stack uses them (GPU): layer norm, a linear
attention layer and an LSTM layer over the same steps, the gradients back through all three, and AdamW on
every weight of the LSTM and the norm.  The gradients are compared with autograd in float64 through the same
equations; the weights with AdamW's formula.

Tolerances: float32 throughout.  The LSTM's gradients are within 1e-4 of their largest value (this library's
bound for it), out within 1e-5; what passes through it carries that further, so the gradients in front of it
are compared at twice that, relative to their largest value.
"""
import pytest
import torch

from layer_lstm_b200 import binding
from layer_lstm_b200.optim import AdamW
from layer_lstm_b200.runner import DeviceProblem
from layer_lstm_b200.workloads import Workload, make_inputs

pytestmark = pytest.mark.gpu

B, T, H, D = 3, 70, 2, 32     # rows, steps, heads, sizes of a head
WIDTH = H * D


class Stack:
    """x -> layer norm -> attention (q = k = v = the normed input's heads) -> LSTM -> out."""

    def __init__(self, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        n = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        self.x, self.weight, self.bias = n(B, T, WIDTH), 1 + 0.1 * n(WIDTH), 0.1 * n(WIDTH)
        self.log_decay = torch.tensor([-0.05, -0.5], device="cuda")
        self.lengths = torch.tensor([T, 33, 64], device="cuda", dtype=torch.int32)
        wl = Workload("block", L=1, D=1, I=WIDTH, H=48, T=T, B=B, dtype="f32", train=True, seed=seed)
        self.lstm = DeviceProblem(make_inputs(wl))
        self.lstm.lengths = self.lengths
        self.norm = binding.make_norm_desc(B * T, WIDTH)
        self.att = binding.make_attention_desc(B, T, H, D, D)
        e = lambda *s: torch.empty(s, device="cuda")  # noqa: E731
        self.y, self.mean, self.rstd = e(B, T, WIDTH), e(B * T), e(B * T)
        self.dq, self.dk, self.dv = e(B, T, H, D), e(B, T, H, D), e(B, T, H, D)
        self.dx, self.dweight, self.dbias = e(B, T, WIDTH), e(WIDTH), e(WIDTH)
        size = max(binding.lstm_layer_norm_workspace_size(self.norm),
                   binding.lstm_linear_attention_workspace_size(self.att))
        self.ws = torch.empty(size, device="cuda", dtype=torch.uint8)   # one after the other on one stream
        params = [self.weight, self.bias] + self.lstm.w_ih + self.lstm.w_hh + self.lstm.b_ih + self.lstm.b_hh
        grads = [self.dweight, self.dbias] + self.lstm.dw_ih + self.lstm.dw_hh + self.lstm.db_ih + self.lstm.db_hh
        self.opt = AdamW(params, grads, lr=1e-2, weight_decay=0.0)

    def step(self, stream=None):
        c = binding.check
        c(binding.lstm_layer_norm_forward(self.norm, self.x, self.weight, self.bias, self.y, self.mean, self.rstd,
                                          stream))
        # the attention's output is the LSTM's input
        c(binding.lstm_linear_attention_forward(self.att, self.y, self.y, self.y, self.log_decay, None, self.lstm.x,
                                                None, self.ws, stream, lengths=self.lengths))
        c(self.lstm.forward(stream))
        c(self.lstm.backward(stream))
        c(binding.lstm_linear_attention_backward(self.att, self.y, self.y, self.y, self.log_decay, None, self.lstm.dx,
                                                 None, self.dq, self.dk, self.dv, None, self.ws, stream,
                                                 lengths=self.lengths))
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            self.dq.add_(self.dk).add_(self.dv)
        c(binding.lstm_layer_norm_backward(self.norm, self.dq, self.x, self.weight, self.mean, self.rstd, self.dx,
                                           self.dweight, self.dbias, self.ws, stream))
        self.opt.step(stream)

    def reference(self):
        """Gradients by autograd in float64: x, norm weight and bias, W_ih, W_hh, bias."""
        leaf = [t.double().clone().requires_grad_() for t in
                (self.x, self.weight, self.bias, self.lstm.w_ih[0], self.lstm.w_hh[0], self.lstm.b_ih[0])]
        x, w, b, wih, whh, bias = leaf
        other = self.lstm.b_hh[0].double()
        y = torch.nn.functional.layer_norm(x, (WIDTH,), w, b, self.norm.eps).view(B, T, H, D)
        g = self.log_decay.double().exp().view(1, H, 1, 1)
        S = torch.zeros(B, H, D, D, device="cuda", dtype=torch.float64)
        h = torch.zeros(B, 48, device="cuda", dtype=torch.float64)
        c = torch.zeros_like(h)
        loss = 0.0
        go = self.lstm.grad_out.double()
        for t in range(T):
            on = (t < self.lengths)[:, None]
            S = torch.where(on[..., None, None], g * S + y[:, t, :, :, None] * y[:, t, :, None, :], S)
            o = (y[:, t, :, None, :] @ S)[:, :, 0].reshape(B, WIDTH) * self.att.scale
            z = o @ wih.t() + h @ whh.t() + bias + other
            i, f, gg, oo = z.chunk(4, 1)
            c = torch.where(on, f.sigmoid() * c + i.sigmoid() * gg.tanh(), c)
            h = torch.where(on, oo.sigmoid() * c.tanh(), h)
            loss = loss + (torch.where(on, h, torch.zeros_like(h)) * go[:, t]).sum()
        return torch.autograd.grad(loss, leaf)


def test_gradients_and_update(cuda_lib):
    s = Stack(21)
    want = s.reference()
    before = [p.clone() for p in s.opt.params]
    s.step()
    binding.check(s.lstm.status())
    got = (s.dx, s.dweight, s.dbias, s.lstm.dw_ih[0], s.lstm.dw_hh[0], s.lstm.db_ih[0])
    for name, a, b in zip(("dx", "dweight", "dbias", "dW_ih", "dW_hh", "db"), got, want):
        assert (a.double() - b).abs().max() <= 2e-4 * b.abs().max(), name
    # the first step of AdamW without decay: lr g / (|g| + eps')
    for p, p0, g in zip(s.opt.params, before, s.opt.grads):
        upd = 1e-2 * g.double() / (g.double().abs() + 1e-8)
        assert (p.double() - (p0.double() - upd)).abs().max() <= 1e-2 * 2.0 ** -19 + 2.0 ** -22 * p0.abs().max()


def test_captured_step_equals_eager_steps(cuda_lib):
    """Three replays of a captured step against three eager steps: the same kernels on the same values."""
    a, b = Stack(22), Stack(22)
    for _ in range(3):
        a.step()
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        b.step(s)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert int(b.opt.state["step"]) == 3
    for p, q in zip(a.opt.params + [a.dx], b.opt.params + [b.dx]):
        assert torch.equal(p, q)


def test_status_word_of_the_shared_workspace(cuda_lib):
    s = Stack(23)
    s.ws.fill_(255)
    binding.check(binding.lstm_linear_attention_forward(s.att, s.x, s.x, s.x, s.log_decay, None, s.y, None, s.ws))
    assert binding.lstm_query_status(s.ws) == binding.LSTM_OK
    d = binding.make_attention_desc(B, T, H, D, D, dtype=binding.LSTM_BF16)
    x, y = s.x.bfloat16(), torch.empty(B, T, H, D, device="cuda", dtype=torch.bfloat16)
    s.ws.fill_(255)
    binding.check(binding.lstm_linear_attention_forward(d, x, x, x, s.log_decay, None, y, None, s.ws))
    assert binding.lstm_query_status(s.ws) == binding.LSTM_OK
    # two calls at once on two streams, a workspace each
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    torch.cuda.synchronize()
    for k, st in enumerate(streams):
        ws, o = torch.empty_like(s.ws), torch.empty_like(y)
        for _ in range(5):
            binding.check(binding.lstm_linear_attention_forward(d, x, x, x, s.log_decay, None, o, None, ws, st))
        outs.append((ws, o))
    torch.cuda.synchronize()
    for _, o in outs:
        assert torch.equal(o, y)

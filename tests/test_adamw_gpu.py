"""lstm_adamw_step against its formula in float64 (GPU).

Tolerances: one step rounds a value of magnitude |x| a few times in float32.
Decoding a code: c / most has the constant's rounding and the product's, 2
half-steps; its square 2 * 2 + 1 = 5, times the scale 6 for m; the square of
that 2 * 5 + 1 = 11, times the scale 12 for v.  m: the decode, two products, a
sum and the rounded coefficients, 6 + 4 = 10 of |b1 m| + |c1 g|; v: 12 + 4 = 16.
p's update: m (10), half of v's 16 and the root (9), the two coefficients and
their products (4), sum and division (2): 25, of the update's magnitude; p itself
3.  A half-step is 2^-24 relative.
"""
import numpy as np
import pytest
import torch

from layer_lstm_b200 import binding
from layer_lstm_b200.optim import BLOCK, AdamW

pytestmark = pytest.mark.gpu

H = 2.0 ** -24
HYPER = dict(lr=3e-3, beta1=0.9, beta2=0.99, eps=1e-8, weight_decay=0.1)


def _tensors(sizes, gdt, seed, offset=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def make(n, std, dt=torch.float32):
        return (torch.randn(n + offset, generator=g, device="cuda") * std).to(dt)[offset:]

    return [make(n, 0.3) for n in sizes], [make(n, 0.02, gdt) for n in sizes]


def _reference(p, g, m, v, t, lr=1.0, gs=1.0):
    """(p, m, v, magnitudes) after step t in float64."""
    h = dict(HYPER)
    rate = h["lr"] * lr
    p, g, m, v = p.double(), g.double() * gs, m.double(), v.double()
    m2 = h["beta1"] * m + (1 - h["beta1"]) * g
    v2 = h["beta2"] * v + (1 - h["beta2"]) * g * g
    upd = rate * (m2 / (1 - h["beta1"] ** t)) / ((v2 / (1 - h["beta2"] ** t)).sqrt() + h["eps"])
    # a moment that cancels keeps the rounding of its terms
    mag = h["beta1"] * m.abs() + (1 - h["beta1"]) * g.abs()
    umag = upd.abs() * torch.where(m2 != 0, mag / m2.abs(), torch.ones_like(mag))
    return p * (1 - rate * h["weight_decay"]) - upd, m2, v2, mag, umag


def _check_step(p0, g, m0, v0, opt, i, t, **kw):
    p, m, v, mag, umag = _reference(p0, g, m0, v0, t, **kw)
    assert ((opt.params[i].double() - p).abs() <= 25 * H * umag + 3 * H * (p0.double().abs() + umag)).all()
    return p, m, v, mag


SIZES = {"one": [1], "ragged": [255, 256, 257, 0, 2047, 2049, 5000], "many": [(7 * i) % 300 for i in range(150)],
         "large": [3_000_001]}


@pytest.mark.parametrize("name", list(SIZES))
@pytest.mark.parametrize("gdt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("offset", [0, 1])
def test_float32_moments(name, gdt, offset, cuda_lib):
    p, g = _tensors(SIZES[name], gdt, 1, offset)
    copies = [torch.zeros(x.numel() + offset, device="cuda", dtype=torch.bfloat16)[offset:] if i % 3 else None
              for i, x in enumerate(p)]
    opt = AdamW(p, g, copies=copies, **HYPER)
    for t in (1, 2, 3):
        before = [[x.clone() for x in ts] for ts in (p, opt.state["m"], opt.state["v"])]
        opt.step()
        for i in range(len(p)):
            _, m, v, mag = _check_step(before[0][i], g[i], before[1][i], before[2][i], opt, i, t)
            assert ((opt.state["m"][i].double() - m).abs() <= 10 * H * mag).all()
            assert ((opt.state["v"][i].double() - v).abs() <= 16 * H * v).all()
            if copies[i] is not None:
                assert torch.equal(copies[i], p[i].to(torch.bfloat16))
        assert int(opt.state["step"]) == t
        for x in g:
            x.mul_(-0.7)


def _words(seed, t, tensor, n):
    """The 32 random bits of each element, in numpy."""
    def pcg(x):
        s = (x * np.uint64(747796405) + np.uint64(2891336453)) & np.uint64(0xFFFFFFFF)
        w = (((s >> ((s >> np.uint64(28)) + np.uint64(4))) ^ s) * np.uint64(277803737)) & np.uint64(0xFFFFFFFF)
        return (w >> np.uint64(22)) ^ w
    u = np.uint64
    k = pcg(u(t & 0xFFFFFFFF) ^ pcg(u(seed & 0xFFFFFFFF) ^ pcg(u(seed >> 32))))
    return pcg(np.arange(n, dtype=np.uint64) ^ pcg(k ^ u(tensor)))


def _decoded(code, scale, power, most):
    a = torch.repeat_interleave(scale.double(), BLOCK)[: code.numel()]
    c = code.double() / most
    return c.sign() * c.abs() ** power * a


def _check_codes(x, err, code, scale, u, power, most):
    """Codes of the float64 values x, which the kernel has within err.  In units of the code's power
    (X = |x| / a most^power) that and the roundings of the scale, its inverse and the products are dX; the
    powers of two neighbouring codes are rounded too.  Within that of a border either code is right."""
    n = x.numel()
    pad = torch.nn.functional.pad
    a = pad(x.abs(), (0, -n % BLOCK)).view(-1, BLOCK).amax(1)
    assert ((scale.double() - a).abs() <= pad(err, (0, -n % BLOCK)).view(-1, BLOCK).amax(1)).all()
    z = torch.repeat_interleave(torch.where(a > 0, 1 / a.clamp(min=1e-300), 0.0), BLOCK)[:n]
    X = (x.abs() * z).clamp(max=1.0) * most ** power
    da = torch.repeat_interleave(pad(err, (0, -n % BLOCK)).view(-1, BLOCK).amax(1), BLOCK)[:n]
    dX = err * z * most ** power + (da * z + 8 * H) * X
    c = torch.floor(X ** (1 / power) * (1 + 1e-12))
    lo, hi = c ** power, (c + 1) ** power
    want = (c + (u * (hi - lo) < X - lo)).clamp(max=most)
    if power == 4:
        want = torch.where(X > 0, want.clamp(min=1), want)
    got = code.double().abs()
    slack = dX + 4 * H * hi
    near = ((X - lo - u * (hi - lo)).abs() <= slack) | ((X - lo).abs() <= slack) | ((hi - X).abs() <= slack)
    assert ((got == want) | (near & ((got - want).abs() <= 1))).all()
    assert ((torch.sign(code.double()) * torch.sign(x) >= 0) | (x.abs() <= err)).all()


@pytest.mark.parametrize("name", list(SIZES))
@pytest.mark.parametrize("gdt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("offset", [0, 1])
def test_eight_bit_moments(name, gdt, offset, cuda_lib):
    seed = 0x1234567890ABCDEF
    p, g = _tensors(SIZES[name], gdt, 2, offset)
    for x in g:
        x[::7] = 0
    opt = AdamW(p, g, state_bits=8, seed=seed, **HYPER)
    st = opt.state
    for t in (1, 2, 3):
        p0 = [x.clone() for x in p]
        m0 = [_decoded(c, s, 2, 127) for c, s in zip(st["m"], st["m_scale"])]
        v0 = [_decoded(c, s, 4, 255) for c, s in zip(st["v"], st["v_scale"])]
        opt.step()
        m_flat, v_flat = opt.read_state()
        at = 0
        for i in range(len(p)):
            n = p[i].numel()
            _, m, v, mag = _check_step(p0[i], g[i], m0[i], v0[i], opt, i, t)
            w = _words(seed, t, i, n)
            um = torch.from_numpy((w & np.uint64(0xFFFF)).astype(np.float64) / 65536).cuda()
            uv = torch.from_numpy((w >> np.uint64(16)).astype(np.float64) / 65536).cuda()
            if n:
                _check_codes(m, 10 * H * mag, st["m"][i], st["m_scale"][i], um, 2, 127)
                _check_codes(v, 16 * H * v, st["v"][i], st["v_scale"][i], uv, 4, 255)
            for flat, code, scale, power, most, steps in ((m_flat, st["m"][i], st["m_scale"][i], 2, 127, 6),
                                                          (v_flat, st["v"][i], st["v_scale"][i], 4, 255, 12)):
                d = _decoded(code, scale, power, most)
                assert ((flat[at:at + n].double() - d).abs() <= steps * H * d.abs()).all()
            at += n
        for x in g:
            x.mul_(-0.7)


def test_eight_bit_rounding_keeps_the_mean(cuda_lib):
    """A second moment far from its gradient's square moves by the step's fraction on average: 2^20 elements
    of one value decay by beta2 a step.  Neighbouring codes are at most 4 / 255 of the scale a apart
    (the slope of x^4 at 1), so the mean over n draws of a rounding of variance at most gap^2 / 4 is off by
    under 5 gap / (2 sqrt(n)); the random 16 bits round down, by up to 2^-16 of a gap."""
    n = 1 << 20
    p, g = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    g[::BLOCK] = 1.0
    opt = AdamW([p], [g], state_bits=8, **HYPER)
    opt.state["v"][0].fill_(100)
    opt.state["v_scale"][0].fill_(1.0)
    opt.step()
    _, v = opt.read_state()
    rest = torch.ones(n, dtype=torch.bool, device="cuda")
    rest[::BLOCK] = False
    want = (100 / 255) ** 4 * 0.99
    a = opt.state["v_scale"][0].double().mean().item()
    gap = 4 / 255 * a
    assert abs(v[rest].double().mean().item() - want) <= 5 * gap / (2 * n ** 0.5) + 2.0 ** -16 * gap + 1e-6 * want


def test_nan_and_tiny_blocks(cuda_lib):
    n = 4 * BLOCK
    p, g = torch.zeros(n, device="cuda"), torch.full((n,), 0.5, device="cuda")
    g[3] = float("nan")
    g[BLOCK + 5] = float("inf")
    g[2 * BLOCK:3 * BLOCK] = 0
    opt = AdamW([p], [g], state_bits=8, **HYPER)
    opt.step()
    m, v = opt.read_state()
    for x in (m, v):
        assert x[:2 * BLOCK].isnan().all()
        assert (x[2 * BLOCK:3 * BLOCK] == 0).all()
        assert (x[3 * BLOCK:] > 0).all()
    assert p[3].isnan() and p[4:BLOCK].isfinite().all() and (p[3 * BLOCK:] < 0).all()


@pytest.mark.parametrize("bits", [8, 32])
def test_graph_counts_steps_and_follows_factors(bits, cuda_lib):
    sizes = [300, 2049]
    runs = []
    for graphed in (False, True):
        p, g = _tensors(sizes, torch.float32, 3)
        factors = torch.tensor([1.0, 1.0], device="cuda")
        opt = AdamW(p, g, state_bits=bits, scalars=factors, **HYPER)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        if graphed:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=s):
                opt.step(stream=s)
        for f in ((1.0, 1.0), (0.5, 2.0), (0.0, 1.0)):
            factors.copy_(torch.tensor(f))
            torch.cuda.synchronize()
            graph.replay() if graphed else opt.step(stream=s)
            torch.cuda.synchronize()
        assert int(opt.state["step"]) == 3
        runs.append(p + opt.state["m"] + opt.state["v"])
    for a, b in zip(*runs):
        assert torch.equal(a, b)


def test_factors_against_formula(cuda_lib):
    p, g = _tensors([1000], torch.float32, 4)
    opt = AdamW(p, g, scalars=torch.tensor([0.25, 3.0], device="cuda"), **HYPER)
    p0 = p[0].clone()
    opt.step()
    zero = torch.zeros_like(p0)
    _check_step(p0, g[0], zero, zero, opt, 0, 1, lr=0.25, gs=3.0)


def test_no_tensors_moves_the_counter(cuda_lib):
    opt = AdamW([], [])
    opt.step()
    assert int(opt.state["step"]) == 1


@pytest.mark.parametrize("dtype,bits", [("f32", 32), ("bf16", 8)])
def test_lstm_training_step_updates_weights(dtype, bits, cuda_lib):
    """dp.train_step with the optimizer of a training problem: the weights move by the formula on the
    gradients the backward wrote, and the layer computes with the moved weights."""
    from layer_lstm_b200.dp import GradBucket, train_step
    from layer_lstm_b200.runner import DeviceProblem
    from layer_lstm_b200.workloads import Workload, make_inputs
    wl = Workload("t", L=2, D=2, I=24, H=40, T=6, B=5, dtype=dtype, state_std=0.3, train=True, seed=77)
    prob = DeviceProblem(make_inputs(wl))
    bucket = GradBucket.adopt(prob, wl.bias)
    opt = prob.optimizer(state_bits=bits, seed=5, **HYPER)
    assert len(opt.params) == 16
    before = [p.clone() for p in opt.params]
    train_step(prob.step, bucket, 1, optimizer=opt)
    binding.check(prob.status())
    out = prob.out.clone()
    for i, p0 in enumerate(before):
        zero = torch.zeros_like(p0)
        _check_step(p0, opt.grads[i], zero, zero, opt, i, 1)
        assert not torch.equal(opt.params[i], p0)
    weights = prob.w_ih + prob.w_hh + prob.b_ih + prob.b_hh
    for w, p in zip(weights, opt.params):
        assert torch.equal(w, p.to(w.dtype))
    binding.check(prob.forward())
    torch.cuda.synchronize()
    assert not torch.equal(out, prob.out)

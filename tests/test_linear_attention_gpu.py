"""lstm_linear_attention_* against the recurrence in float64, gradients by autograd through it (GPU).

Tolerances, relative to the sum of the magnitudes of a value's terms (the same
recurrence on absolute values).  Float32: a term passes N = 2 max(dk, dv) + 256
+ T / 8 roundings at most (a product over dk, one over a chunk, a decay and a
sum per chunk, 4 for an exponential), each half a step H = 2^-24, and a decay
exp(x) of up to 64 steps adds |x| half-steps from its argument, at most 100 for
the decays used here.  bf16: the score and the state enter the products
rounded (2^-8 of their magnitudes, between them every term once), the result
is rounded once (2^-8 of it); the states' weighted keys keep 2^-16.
"""
import itertools

import pytest
import torch

from layer_lstm_b200 import binding

pytestmark = pytest.mark.gpu

H32 = 2.0 ** -24
HB = 2.0 ** -8


def _reference(q, k, v, ld, s0, lengths, scale, grads=None):
    """(B, T, H, .) float64 arrays -> out, s_n, and with grads (grad_out, grad_sn) the gradients."""
    leaf = [t.clone().requires_grad_(grads is not None) for t in (q, k, v, s0)]
    q, k, v, S = leaf
    B, T = q.shape[:2]
    g = ld.clamp(-1e4, 0).exp().view(1, -1, 1, 1)
    outs = []
    for t in range(T):
        on = (t < lengths).view(B, 1, 1, 1)
        new = g * S + k[:, t, :, :, None] * v[:, t, :, None, :]
        S = torch.where(on, new, S)
        o = scale * (q[:, t, :, None, :] @ S)[:, :, 0]
        outs.append(torch.where(on[..., 0], o, torch.zeros_like(o)))
    out = torch.stack(outs, 1) if outs else torch.zeros(B, 0, *v.shape[2:], device=v.device, dtype=v.dtype)
    if grads is None:
        return [out, S]
    loss = (S * grads[1]).sum() + (out * grads[0]).sum()
    gr = torch.autograd.grad(loss, leaf, allow_unused=True, materialize_grads=True)
    return [out.detach(), S.detach(), *gr]


def _inputs(B, T, H, dk, dv, dt, seed, ragged, batch_first=True, packed=False):
    g = torch.Generator(device="cuda").manual_seed(seed)
    lead = (B, T) if batch_first else (T, B)

    def n(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    if packed:
        row = H * (2 * dk + dv)
        p = n(*lead, row).to(dt)
        q, k, v = (p[..., a:a + H * w].view(*lead, H, w) for a, w in ((0, dk), (H * dk, dk), (2 * H * dk, dv)))
    else:
        row = 0
        q, k, v = n(*lead, H, dk).to(dt), n(*lead, H, dk).to(dt), n(*lead, H, dv).to(dt)
    lengths = None
    if ragged:
        lengths = torch.randint(0, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        lengths[0] = T + 5      # clamped
        if B > 1:
            lengths[1] = 0
        if B > 2:
            lengths[2] = -3
    # memories of 4 to 250 steps and one head without decay
    ld = torch.log1p(-torch.exp2(-2 - 6 * torch.rand(H, generator=g, device="cuda")))
    ld[H // 2] = 0.0
    s0, gs = n(B, H, dk, dv), n(B, H, dk, dv)
    go = n(*lead, H, dv).to(dt)
    return dict(q=q, k=k, v=v, ld=ld, s0=s0, gs=gs, go=go, lengths=lengths, row=row)


def _desc(t, B, T, H, dk, dv, dt, batch_first=True, scale=None):
    return binding.make_attention_desc(B, T, H, dk, dv, batch_first,
                                       binding.LSTM_F32 if dt == torch.float32 else binding.LSTM_BF16, scale,
                                       t["row"], t["row"], t["row"])


def _run(t, d, dt, with_s0=True, with_gs=True, poison=True, stream=None):
    B, H, dk, dv = d.batch, d.heads, d.key_size, d.value_size
    ws = torch.full((binding.lstm_linear_attention_workspace_size(d),), 255, device="cuda", dtype=torch.uint8)
    q, k, v, go = t["q"], t["k"], t["v"], t["go"]
    if t["lengths"] is not None and poison:    # what lies at padded steps is never read
        T = d.seq_len
        pad = torch.arange(T, device="cuda")[None] >= t["lengths"][:, None]
        if not d.batch_first:
            pad = pad.t()
        for x in (q, k, v, go):
            x[pad] = float("nan")
    full = lambda x: torch.full_like(x, 7.0) if x.is_contiguous() else x.clone(memory_format=torch.preserve_format)  # noqa: E731
    out, s_n = torch.full_like(go, 7.0), torch.full((B, H, dk, dv), 7.0, device="cuda")
    s0, gs = t["s0"] if with_s0 else None, t["gs"] if with_gs else None
    binding.check(binding.lstm_linear_attention_forward(d, q, k, v, t["ld"], s0, out, s_n, ws, lengths=t["lengths"],
                                                        stream=stream))
    if t["row"]:
        p = torch.full((*q.shape[:2], t["row"]), 7.0, device="cuda", dtype=dt)
        dq, dk_, dv_ = (p[..., a:a + H * w].view(*q.shape[:2], H, w)
                        for a, w in ((0, dk), (H * dk, dk), (2 * H * dk, dv)))
    else:
        dq, dk_, dv_ = full(q), full(k), full(v)
    ds0 = torch.full((B, H, dk, dv), 7.0, device="cuda")
    binding.check(binding.lstm_linear_attention_backward(d, q, k, v, t["ld"], s0, go, gs, dq, dk_, dv_, ds0, ws,
                                                         lengths=t["lengths"], stream=stream))
    return [out, s_n, dq, dk_, dv_, ds0]


def _check(t, d, dt, got, with_s0=True, with_gs=True):
    bf = d.batch_first
    B, T = d.batch, d.seq_len
    n = t["lengths"] if t["lengths"] is not None else torch.full((B,), T, device="cuda", dtype=torch.int32)
    n = n.clamp(0, T)
    pad = (torch.arange(T, device="cuda")[None] >= n[:, None])[..., None, None]

    def lead(x):
        x = (x if bf else x.transpose(0, 1)).double()
        return torch.where(pad, torch.zeros_like(x), x)

    a = [lead(t[x]) for x in "qkv"] + [t["ld"].double()]
    s0 = t["s0"].double() * (1.0 if with_s0 else 0.0)
    gr = (lead(t["go"]), t["gs"].double() * (1.0 if with_gs else 0.0))
    ref = _reference(*a, s0, n, d.scale, gr)
    mag = _reference(*(x.abs() for x in a[:3]), a[3], s0.abs(), n, abs(d.scale), [x.abs() for x in gr])
    N = 2 * max(d.key_size, d.value_size) + 256 + T / 8 + 100
    # forward order: out, s_n, then dq, dk, dv, ds0
    for i, (name, x) in enumerate(zip(("out", "s_n", "dq", "dk", "dv", "ds0"), got)):
        state = name in ("s_n", "ds0")
        y = x.double() if state or bf else x.double().transpose(0, 1)
        tol = N * H32 * mag[i]
        if dt == torch.bfloat16:
            tol = tol + (2.0 ** -16 * mag[i] if state else HB * mag[i] + HB * ref[i].abs() * (1 + HB))
        err = (y - ref[i]).abs()
        assert (err <= tol).all(), (name, (err - tol).max().item(), (err / tol.clamp(min=1e-300)).max().item())
        if not state:
            assert (y[pad.expand_as(y)] == 0).all(), name


DIMS = [(64, 64), (128, 128), (32, 32), (16, 16), (1, 1), (40, 72), (128, 64), (64, 128), (96, 33), (17, 128), (48, 80)]
TIMES = [1, 2, 63, 64, 65, 127, 128, 129, 200, 333]


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dk,dv", DIMS)
def test_sizes(dk, dv, dt, cuda_lib):
    for i, T in enumerate(TIMES if dk == dv else (1, 64, 131)):
        B, H = (3, 2) if i % 2 else (2, 3)
        for ragged in (False, True):
            t = _inputs(B, T, H, dk, dv, dt, 10 * i + ragged, ragged)
            d = _desc(t, B, T, H, dk, dv, dt)
            _check(t, d, dt, _run(t, d, dt))


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("batch_first,packed,with_s0,with_gs",
                         [c for c in itertools.product((True, False), repeat=4) if not all(c[::2])])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (24, 40)])
def test_layouts(dk, dv, batch_first, packed, with_s0, with_gs, dt, cuda_lib):
    B, T, H = 4, 150, 2
    t = _inputs(B, T, H, dk, dv, dt, 3, True, batch_first, packed)
    d = _desc(t, B, T, H, dk, dv, dt, batch_first, scale=-0.3)
    _check(t, d, dt, _run(t, d, dt, with_s0, with_gs), with_s0, with_gs)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,T,H,dk,dv", [(1, 1500, 1, 64, 64), (2, 1111, 2, 128, 128), (1, 2049, 3, 32, 32),
                                         (2, 900, 1, 20, 36)])
def test_long_sequences(B, T, H, dk, dv, dt, cuda_lib):
    """Few rows and heads: the time axis is cut into segments."""
    for ragged in (False, True):
        t = _inputs(B, T, H, dk, dv, dt, 4, ragged)
        d = _desc(t, B, T, H, dk, dv, dt)
        _check(t, d, dt, _run(t, d, dt))


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_many_heads(dt, cuda_lib):
    t = _inputs(40, 70, 16, 64, 64, dt, 5, True)
    d = _desc(t, 40, 70, 16, 64, 64, dt)
    _check(t, d, dt, _run(t, d, dt))


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_extreme_decays(dt, cuda_lib):
    """Decays that forget at once, within a chunk, hardly or (clamped) never."""
    B, T, H, dk, dv = 2, 200, 6, 64, 64
    t = _inputs(B, T, H, dk, dv, dt, 6, False)
    t["ld"].copy_(torch.tensor([float("-inf"), -50.0, -1.5, -1e-6, 0.0, 3.0]))
    d = _desc(t, B, T, H, dk, dv, dt)
    _check(t, d, dt, _run(t, d, dt))


def test_no_steps_and_in_place_state(cuda_lib):
    t = _inputs(2, 0, 3, 16, 24, torch.float32, 7, False)
    d = _desc(t, 2, 0, 3, 16, 24, torch.float32)
    got = _run(t, d, torch.float32)
    assert torch.equal(got[1], t["s0"]) and torch.equal(got[5], t["gs"])
    for T in (100, 3000):
        t = _inputs(1, T, 2, 64, 64, torch.float32, 8, False)
        d = _desc(t, 1, T, 2, 64, 64, torch.float32)
        want = _run(t, d, torch.float32)[1]
        ws = torch.empty(binding.lstm_linear_attention_workspace_size(d), device="cuda", dtype=torch.uint8)
        s, out = t["s0"].clone(), torch.empty_like(t["go"])
        binding.check(binding.lstm_linear_attention_forward(d, t["q"], t["k"], t["v"], t["ld"], s, out, s, ws))
        assert torch.equal(s, want)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,H,dk,dv", [(1, 1, 1, 1), (3, 2, 64, 64), (5, 3, 128, 128), (2, 2, 40, 72), (4, 3, 17, 33),
                                       (600, 4, 32, 32), (2, 1, 100, 6)])
def test_step_is_one_token_of_the_forward(B, H, dk, dv, dt, cuda_lib):
    for ragged in (False, True):
        t = _inputs(B, 1, H, dk, dv, dt, 9, ragged)
        if ragged:
            t["lengths"] = (torch.arange(B, device="cuda") % 3 - 1).int().clamp(max=1)
        d = _desc(t, B, 1, H, dk, dv, dt)
        state, out = t["s0"].clone(), torch.full_like(t["go"], 7.0)
        binding.check(binding.lstm_linear_attention_step(d, t["q"], t["k"], t["v"], t["ld"], state, out,
                                                         lengths=t["lengths"]))
        n = t["lengths"].clamp(0, 1) if ragged else torch.ones(B, device="cuda", dtype=torch.int32)
        a = [t[x].double() for x in "qkv"] + [t["ld"].double(), t["s0"].double(), n]
        ref = _reference(*a, d.scale)
        mag = _reference(*(x.abs() for x in a[:3]), a[3], a[4].abs(), n, d.scale)
        assert ((state.double() - ref[1]).abs() <= 8 * H32 * mag[1]).all()
        tol = (dk + 12) * H32 * mag[0] + (HB * ref[0].abs() * (1 + HB) if dt == torch.bfloat16 else 0)
        assert ((out.double() - ref[0]).abs() <= tol).all()
        if ragged:
            assert torch.equal(state[n == 0], t["s0"][n == 0]) and (out[n == 0] == 0).all()


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_prompt_then_tokens(dt, cuda_lib):
    """A prompt's state carried on by single steps gives the whole sequence's outputs and state."""
    B, T, H, dk, dv = 2, 90, 3, 64, 64
    t = _inputs(B, T, H, dk, dv, dt, 11, False)
    d = _desc(t, B, T, H, dk, dv, dt)
    whole = _run(t, d, dt)
    P = 77
    dp, d1 = _desc(t, B, P, H, dk, dv, dt), _desc(t, B, 1, H, dk, dv, dt)
    ws = torch.empty(binding.lstm_linear_attention_workspace_size(dp), device="cuda", dtype=torch.uint8)
    s, out = torch.empty_like(t["s0"]), torch.empty_like(t["go"][:, :P].contiguous())
    binding.check(binding.lstm_linear_attention_forward(dp, *(t[x][:, :P].contiguous() for x in "qkv"), t["ld"],
                                                        t["s0"], out, s, ws))
    outs = [out]
    for i in range(P, T):
        o = torch.empty_like(t["go"][:, i].contiguous())
        binding.check(binding.lstm_linear_attention_step(d1, *(t[x][:, i].contiguous() for x in "qkv"), t["ld"], s, o))
        outs.append(o[:, None])
    got = torch.cat(outs, 1)
    # both sides are within the forward's tolerance of the recurrence, whose largest values are near 100
    bound = 3e-2 if dt == torch.bfloat16 else 1e-4
    assert (got.double() - whole[0].double()).abs().max() <= bound * whole[0].double().abs().max()
    assert (s - whole[1]).abs().max() <= 1e-4 * whole[1].abs().max()


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,T,H", [(4, 100, 3), (1, 1600, 1)])
def test_graph_replay_and_repeat(B, T, H, dt, cuda_lib):
    """A captured forward and backward, replayed, gives what the eager calls gave, bit for bit."""
    t = _inputs(B, T, H, 64, 64, dt, 12, True)
    d = _desc(t, B, T, H, 64, 64, dt)
    eager = _run(t, d, dt)
    again = _run(t, d, dt)
    for a, b in zip(eager, again):
        assert torch.equal(a, b)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    ws = torch.empty(binding.lstm_linear_attention_workspace_size(d), device="cuda", dtype=torch.uint8)
    out = [torch.zeros_like(x) for x in eager]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        binding.check(binding.lstm_linear_attention_forward(d, t["q"], t["k"], t["v"], t["ld"], t["s0"], out[0],
                                                            out[1], ws, lengths=t["lengths"], stream=s))
        binding.check(binding.lstm_linear_attention_backward(d, t["q"], t["k"], t["v"], t["ld"], t["s0"], t["go"],
                                                             t["gs"], out[2], out[3], out[4], out[5], ws,
                                                             lengths=t["lengths"], stream=s))
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    for a, b in zip(eager, out):
        assert torch.equal(a, b)


def test_gradients_against_differences(cuda_lib):
    """The loss along one direction of every input, central differences of the library's own forward in
    float32: step 1e-2 on a function that is at most cubic along a line, so the difference is off by the
    third-order term (h^2 of the value's size) and the forward's rounding over h: 1e-3 of the terms' size."""
    B, T, H, dk, dv = 2, 70, 2, 32, 48
    t = _inputs(B, T, H, dk, dv, torch.float32, 13, False)
    d = _desc(t, B, T, H, dk, dv, torch.float32)
    got = _run(t, d, torch.float32)
    u = {x: torch.randn_like(t[x]) for x in ("q", "k", "v", "s0")}
    ws = torch.empty(binding.lstm_linear_attention_workspace_size(d), device="cuda", dtype=torch.uint8)

    def loss(h):
        out, s_n = torch.empty_like(t["go"]), torch.empty_like(t["s0"])
        a = {x: t[x] + h * u[x] for x in u}
        binding.check(binding.lstm_linear_attention_forward(d, a["q"], a["k"], a["v"], t["ld"], a["s0"], out, s_n, ws))
        return (out.double() * t["go"].double()).sum().item() + (s_n.double() * t["gs"].double()).sum().item()

    parts = [g.double() * u[x].double() for g, x in zip((got[2], got[3], got[4], got[5]), ("q", "k", "v", "s0"))]
    want = sum(p.sum().item() for p in parts)
    size = sum(p.abs().sum().item() for p in parts)
    assert abs((loss(1e-2) - loss(-1e-2)) / 2e-2 - want) <= 1e-3 * size


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dk,dv", [(64, 64), (48, 80), (16, 32), (128, 128), (20, 36)])
def test_heads_and_rows_do_not_mix(dk, dv, dt, cuda_lib):
    """NaN in one head of one row leaves every other head and row as it is, bit for bit."""
    B, T, H = 3, 150, 4
    t = _inputs(B, T, H, dk, dv, dt, 15, False)
    d = _desc(t, B, T, H, dk, dv, dt)
    clean = _run(t, d, dt)
    for x in ("q", "k", "v", "go"):
        t[x][1, :, 2] = float("nan")
    t["s0"][1, 2] = float("nan")
    got = _run(t, d, dt)
    keep = torch.ones(B, H, dtype=torch.bool, device="cuda")
    keep[1, 2] = False
    for name, a, b in zip(("out", "s_n", "dq", "dk", "dv", "ds0"), clean, got):
        if name not in ("s_n", "ds0"):
            a, b = a.transpose(1, 2), b.transpose(1, 2)
        assert torch.equal(a[keep], b[keep]), name
        assert b[1, 2].isnan().any(), name


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_other_stream_and_guard_bytes(dt, cuda_lib):
    """A call on a stream of its own; what lies around the outputs stays."""
    B, T, H, dk, dv = 2, 200, 2, 64, 64
    t = _inputs(B, T, H, dk, dv, dt, 16, True)
    d = _desc(t, B, T, H, dk, dv, dt)
    want = _run(t, d, dt)
    s = torch.cuda.Stream()
    pad = 512
    bufs = [torch.full((x.numel() + 2 * pad,), 3.0, device="cuda", dtype=x.dtype) for x in want]
    o = [b[pad:-pad].view(x.shape) for b, x in zip(bufs, want)]
    ws = torch.empty(binding.lstm_linear_attention_workspace_size(d), device="cuda", dtype=torch.uint8)
    torch.cuda.synchronize()
    binding.check(binding.lstm_linear_attention_forward(d, t["q"], t["k"], t["v"], t["ld"], t["s0"], o[0], o[1], ws,
                                                        lengths=t["lengths"], stream=s))
    binding.check(binding.lstm_linear_attention_backward(d, t["q"], t["k"], t["v"], t["ld"], t["s0"], t["go"],
                                                         t["gs"], o[2], o[3], o[4], o[5], ws, lengths=t["lengths"],
                                                         stream=s))
    s.synchronize()
    for x, y, b in zip(want, o, bufs):
        assert torch.equal(x, y)
        assert (b[:pad] == 3.0).all() and (b[-pad:] == 3.0).all()

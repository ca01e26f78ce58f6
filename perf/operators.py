"""What the sequence-model operators next to the LSTM are measured on.

Three operators a user of this library trains and serves with beside the LSTM
layers: linear attention with a decay for each head (a recurrence with a
matrix state; chunked over sequences, its backward pass, and one step for
single tokens), layer norm (forward and backward), and an AdamW step over
every tensor of a model (states in 32 or in 8 bits).

`run` computes them in elementary torch operations where `own` is false and
through the library's binding where it is true.  Sizes follow the workloads of
layer_lstm_b200/workloads.py (c1 20 rows of 16; c2/c5 64 x 128 steps of 512;
c3 32 x 256 steps of 1024, two directions; c4 batch 512 of 1024) and spread
around them.
"""
import math

import torch

own = False

BLOCK = 256   # elements that share one scale in the 8-bit optimiser states


# ------------------------------------------------------------------ the cases
def listed():
    att = dict(op="att", s0=True, ragged=False, batch_first=True)
    return [
        # one generated token of one stream, 512 wide: latency
        dict(name="att_step_1", op="att_step", dtype="bf16", B=1, H=8, dk=64, dv=64),
        # one generated token for c4's batch of 512, 1024 wide: reads and writes 268 MB of state
        dict(name="att_step_512", op="att_step", dtype="bf16", B=512, H=8, dk=128, dv=128),
        # prompts of c3's shape, 1024 wide, a carried state
        dict(att, name="att_prompt_c3", dtype="bf16", B=32, T=256, H=8, dk=128, dv=128, train=False),
        # one long document, an odd length, no carried state: parallel only over heads and time
        dict(att, name="att_long", dtype="bf16", B=1, T=32767, H=16, dk=64, dv=64, train=False, s0=False),
        # padded batch in float32, time-major, sizes that no tile divides
        dict(att, name="att_odd_f32", dtype="f32", B=5, T=331, H=3, dk=40, dv=72, train=False, ragged=True,
             batch_first=False),
        # training step of c5's shape in float32, 512 wide
        dict(att, name="att_train_c5", dtype="f32", B=64, T=128, H=8, dk=64, dv=64, train=True),
        # training step of c3's shape in bf16, 1024 wide, padded batch
        dict(att, name="att_train_c3", dtype="bf16", B=32, T=256, H=8, dk=128, dv=128, train=True, ragged=True),
        # the output of c1 (4 x 5 steps of 16): latency
        dict(name="norm_c1", op="norm", dtype="f32", rows=20, cols=16, train=False),
        # training step over c5's layer output
        dict(name="norm_train_c5", op="norm", dtype="f32", rows=8192, cols=512, train=True),
        # training step over c3's layer output, both directions
        dict(name="norm_train_c3", op="norm", dtype="bf16", rows=8192, cols=2048, train=True),
        # c5's weights and biases
        dict(name="adamw_c5", op="adamw", bits=32, copy=False, grad="f32", L=2, D=1, I=256, H=512),
        # c3's weights and biases: float32 masters, bf16 copies for the layers, 8-bit states
        dict(name="adamw_c3_8bit", op="adamw", bits=8, copy=True, grad="f32", L=2, D=2, I=512, H=1024),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["att_step", "att", "att", "att_train", "norm", "norm_train", "adamw32", "adamw8"])
    dtype = rng.choice(["f32", "bf16", "bf16"])
    if op.startswith("att"):
        if rng.random() < 0.6:
            dk = dv = rng.choice([32, 64, 128])
        else:
            dk, dv = rng.randint(8, 128), rng.randint(8, 128)
        H = rng.randint(1, 16)
        if op == "att_step":
            return dict(op="att_step", dtype=dtype, B=_log(rng, 1, 512 * 8 // H), H=H, dk=dk, dv=dv)
        most = 16384 if op == "att_train" else 131072          # token-heads of a 128-wide head
        room = int(most * 256 / (dk + dv) / H * (1 if dtype == "bf16" else 0.25))
        T = _log(rng, 1, min(32768, room))
        B = _log(rng, 1, max(1, min(64, room // T)))
        return dict(op="att", dtype=dtype, B=B, T=T, H=H, dk=dk, dv=dv, train=op == "att_train",
                    s0=rng.random() < 0.6, ragged=rng.random() < 0.5, batch_first=rng.random() < 0.6)
    if op.startswith("norm"):
        cols = _log(rng, 16, 4096) if rng.random() < 0.4 else 2 ** rng.randint(4, 12)
        rows = _log(rng, 1, min(65536, (8192 * 2048) // cols))
        return dict(op="norm", dtype=dtype, rows=rows, cols=cols, train=op == "norm_train")
    H = _log(rng, 16, 1024)
    return dict(op="adamw", bits=8 if op == "adamw8" else 32, copy=rng.random() < 0.5,
                grad=rng.choice(["f32", "f32", "bf16"]), L=rng.randint(1, 2), D=rng.randint(1, 2),
                I=_log(rng, 8, 512), H=H)


# ------------------------------------------------------------------ the inputs
def _dt(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _shapes(case):
    """The shapes of an LSTM stack's weights and biases, in its own order."""
    out = []
    for layer in range(case["L"]):
        for _ in range(case["D"]):
            G = 4 * case["H"]
            fan = case["I"] if layer == 0 else case["D"] * case["H"]
            out += [(G, fan), (G, case["H"]), (G,), (G,)]
    return out


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, dtype=torch.float32, std=1.0):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

    def empty(*shape, dtype=torch.float32):
        return torch.zeros(shape, device="cuda", dtype=dtype)

    s = {"case": case}
    if case["op"] in ("att", "att_step"):
        dt, B, H, dk, dv = _dt(case), case["B"], case["H"], case["dk"], case["dv"]
        T = case.get("T", 1)
        lead = (B, T) if case.get("batch_first", True) else (T, B)
        # slow and fast heads: memories of 8 to 1024 steps
        n = torch.arange(H, device="cuda", dtype=torch.float32) / max(1, H - 1)
        s["log_decay"] = torch.log1p(-torch.exp2(-3.0 - 7.0 * n))
        s["q"] = normal(*lead, H, dk, dtype=dt)
        s["k"] = normal(*lead, H, dk, dtype=dt)
        s["v"] = normal(*lead, H, dv, dtype=dt)
        s["out"] = empty(*lead, H, dv, dtype=dt)
        if case["op"] == "att_step":
            s["state"] = normal(B, H, dk, dv, std=2.0)
            return s
        s["s0"] = normal(B, H, dk, dv, std=2.0) if case["s0"] else None
        s["s_n"] = empty(B, H, dk, dv)
        s["lengths"] = None
        if case["ragged"]:
            n = torch.randint(0, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
            n[0] = T
            s["lengths"] = n
        if case["train"]:
            s["grad_out"] = normal(*lead, H, dv, dtype=dt)
            s["grad_sn"] = normal(B, H, dk, dv, std=0.1)
            for a in ("q", "k", "v"):
                s["d" + a] = torch.zeros_like(s[a])
            s["ds0"] = empty(B, H, dk, dv)
    elif case["op"] == "norm":
        dt, R, C = _dt(case), case["rows"], case["cols"]
        s["x"] = (normal(R, C, std=0.5) + normal(R, 1, std=0.2)).to(dt)
        s["weight"], s["bias"] = (1 + normal(C, std=0.1)).to(dt), normal(C, std=0.1, dtype=dt)
        s["y"], s["mean"], s["rstd"] = empty(R, C, dtype=dt), empty(R), empty(R)
        if case["train"]:
            s["grad_y"] = normal(R, C, dtype=dt)
            s["dx"], s["dweight"], s["dbias"] = empty(R, C, dtype=dt), empty(C), empty(C)
    else:
        shapes = _shapes(case)
        gdt = torch.float32 if case["grad"] == "f32" else torch.bfloat16
        bound = 1 / math.sqrt(case["H"])
        s["hyper"] = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01)
        s["seed"] = seed
        s["p"] = [(torch.rand(z, generator=g, device="cuda") * 2 - 1) * bound for z in shapes]
        s["copy"] = [p.to(torch.bfloat16) for p in s["p"]] if case["copy"] else None
        s["g"] = [normal(*z, std=0.01, dtype=gdt) for z in shapes]
        s["step"] = torch.tensor([1000], device="cuda", dtype=torch.int64)
        m = [normal(*z, std=0.003) for z in shapes]
        v = [normal(*z, std=0.01).square() for z in shapes]
        if case["bits"] == 32:
            s["m"], s["v"] = m, v
        else:
            zero = [torch.zeros_like(t, dtype=torch.int64) for t in m]
            mc = [_encode(t, r, 2, 127.0) for t, r in zip(m, zero)]
            vc = [_encode(t, r, 4, 255.0) for t, r in zip(v, zero)]
            s["m"], s["m_scale"] = [c.to(torch.int8) for c, _ in mc], [a for _, a in mc]
            s["v"], s["v_scale"] = [c.to(torch.uint8) for c, _ in vc], [a for _, a in vc]
            total = sum(p.numel() for p in s["p"])
            s["m_out"], s["v_out"] = empty(total), empty(total)
    return s


# ------------------------------------------------------------- the plain forms
def _heads_first(x, batch_first):
    return (x.permute(0, 2, 1, 3) if batch_first else x.permute(1, 2, 0, 3)).float()


def _back(x, batch_first, dtype):
    return (x.permute(0, 2, 1, 3) if batch_first else x.permute(2, 0, 1, 3)).to(dtype).contiguous()


def _mix(a, b, c, ld, reverse=False):
    """sum over j <= i (j >= i when reverse) of exp(ld |i - j|) (a_i . b_j) c_j for (B, H, T, .)
    arrays, in chunks of 64: inside a chunk by its score matrix, across chunks by each chunk's sum of
    b^T c and a triangular matrix of decays over the chunks."""
    if reverse:
        return _mix(a.flip(2), b.flip(2), c.flip(2), ld).flip(2)
    B, H, T, _ = a.shape
    C = 64
    n = -(-T // C)

    def cut(x):
        return torch.nn.functional.pad(x, (0, 0, 0, n * C - T)).view(B, H, n, C, x.shape[3])

    a, b, c = cut(a), cut(b), cut(c)
    i = torch.arange(C, device=a.device, dtype=torch.float32)
    ldh = ld.view(H, 1, 1)
    inside = torch.exp(ldh * (i[:, None] - i[None, :]).clamp(min=0)) * (i[:, None] >= i[None, :])
    out = (a @ b.transpose(3, 4) * inside[None, :, None]) @ c
    if n > 1:
        w = torch.exp(ldh * (C - 1 - i)[None, :, None])
        sums = (b * w[None, :, None]).transpose(3, 4) @ c                       # (B, H, n, da, dc)
        r = torch.arange(n, device=a.device, dtype=torch.float32)
        far = torch.exp(ldh * C * (r[:, None] - 1 - r[None, :]).clamp(min=0)) * (r[:, None] > r[None, :])
        before = (far[None] @ sums.flatten(3)).view_as(sums)
        out = out + (a * torch.exp(ldh * (i + 1)[None, :, None])[None, :, None]) @ before
    return out.reshape(B, H, n * C, out.shape[4])[:, :, :T]


def _att_plain(s):
    case, dt = s["case"], s["q"].dtype
    bf, scale = case["batch_first"], case["dk"] ** -0.5
    q, k, v = (_heads_first(s[a], bf) for a in ("q", "k", "v"))
    B, H, T, dk = q.shape
    ld = s["log_decay"]
    t = torch.arange(T, device=q.device)
    n = s["lengths"].long() if s["lengths"] is not None else torch.full((B,), T, device=q.device)
    valid = (t[None] < n[:, None])[:, None, :, None]
    zero = torch.zeros((), device=q.device)
    q, k, v = (torch.where(valid, x, zero) for x in (q, k, v))
    since = torch.exp(ld[None, :, None] * (t + 1)[None, None])[..., None]                     # decay since s0
    left = torch.where(valid, torch.exp(ld[None, :, None] * (n[:, None, None] - 1 - t[None, None]).clamp(min=0))[..., None],
                       zero)                                                            # decay until s_n
    whole = torch.exp(ld[None] * n[:, None])[..., None, None]
    out = _mix(q, k, v, ld)
    s_n = (k * left).transpose(2, 3) @ v
    if s["s0"] is not None:
        out = out + (q * since) @ s["s0"]
        s_n = s_n + whole * s["s0"]
    res = {"out": _back(torch.where(valid, out * scale, zero), bf, dt), "s_n": s_n}
    if not case["train"]:
        return res
    do = torch.where(valid, _heads_first(s["grad_out"], bf), zero) * scale
    gs = s["grad_sn"]
    dq = _mix(do, v, k, ld)
    ds0 = whole * gs + (q * since).transpose(2, 3) @ do
    if s["s0"] is not None:
        dq = dq + (do * since) @ s["s0"].transpose(2, 3)
    dk = _mix(v, do, q, ld, reverse=True) + (v * left) @ gs.transpose(2, 3)
    dv = _mix(k, q, do, ld, reverse=True) + (k * left) @ gs
    for name, x in (("dq", dq), ("dk", dk), ("dv", dv)):
        res[name] = _back(torch.where(valid, x, zero), bf, dt)
    res["ds0"] = ds0
    return res


def _step_plain(s):
    case = s["case"]
    q, k, v = (s[a][:, 0].float() for a in ("q", "k", "v"))
    g = torch.exp(s["log_decay"])[None, :, None, None]
    s["state"].copy_(s["state"] * g + k[..., :, None] * v[..., None, :])
    out = (q[..., None, :] @ s["state"])[..., 0, :] * case["dk"] ** -0.5
    return {"out": out.to(s["q"].dtype)[:, None], "state": s["state"]}


def _norm_plain(s):
    x, w, b = s["x"].float(), s["weight"].float(), s["bias"].float()
    mean = x.mean(1, keepdim=True)
    d = x - mean
    rstd = torch.rsqrt(d.square().mean(1, keepdim=True) + 1e-5)
    xhat = d * rstd
    res = {"y": (xhat * w + b).to(s["x"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}
    if s["case"]["train"]:
        gy = s["grad_y"].float()
        gx = gy * w
        dx = rstd * (gx - gx.mean(1, keepdim=True) - xhat * (gx * xhat).mean(1, keepdim=True))
        res.update(dx=dx.to(s["x"].dtype), dweight=(gy * xhat).sum(0), dbias=gy.sum(0))
    return res


def _pcg(x):
    """A permutation of 32-bit words (Jarzynski and Olano 2020), on int64 tensors or whole numbers."""
    s = (x * 747796405 + 2891336453) & 0xFFFFFFFF
    w = (((s >> ((s >> 28) + 4)) ^ s) * 277803737) & 0xFFFFFFFF
    return (w >> 22) ^ w


def _blocks(x):
    n = x.numel()
    return torch.nn.functional.pad(x.reshape(-1), (0, -n % BLOCK)).view(-1, BLOCK)


def _encode(x, u16, power, most):
    """8-bit codes of x in blocks of 256 that share their largest magnitude a: code c stands for
    sign(x) (c / most)^power a.  Rounds up with the probability that keeps the value's mean, by u16
    (random whole numbers in [0, 2^16)); a nonzero value of a power of 4 keeps a code of at least 1."""
    y, u = _blocks(x), _blocks(u16).to(torch.float32) * 2.0 ** -16
    mag = y.abs()
    a = mag.amax(1, keepdim=True)
    fine = torch.isfinite(a)
    some = fine & (a >= 2.0 ** -126)
    inv = torch.reciprocal(torch.where(some, a, torch.ones_like(a)))
    z = torch.where(some, mag * inv, torch.zeros_like(mag)).clamp(max=1.0) * most ** power
    c = torch.sqrt(z)
    if power == 4:
        c = torch.sqrt(c)
    c = torch.floor(c)
    lo, hi = c * c, (c + 1) * (c + 1)
    if power == 4:
        lo, hi = lo * lo, hi * hi
    c = torch.where(u * (hi - lo) < z - lo, c + 1, c).clamp(max=most)
    if power == 4:
        c = torch.where(z > 0, c.clamp(min=1.0), c)
    else:
        c = torch.where(y < 0, -c, c)
    scale = torch.where(fine, torch.where(some, a, torch.zeros_like(a)), torch.full_like(a, float("nan")))
    return c.view(-1)[: x.numel()].view(x.shape), scale[:, 0].contiguous()


def _decode(code, scale, power, most):
    c = _blocks(code.to(torch.float32)) * torch.tensor(1.0 / most, dtype=torch.float32, device=code.device)
    x = c.abs() * c if power == 2 else (c * c) * (c * c)
    return (x * scale[:, None]).view(-1)[: code.numel()].view(code.shape)


def _adamw_plain(s):
    h, dev = s["hyper"], s["step"].device
    s["step"] += 1
    t = s["step"].double()
    f = lambda x: torch.as_tensor(x, dtype=torch.float32, device=dev)
    b1, b2, c1, c2 = f(h["beta1"]), f(h["beta2"]), f(1 - h["beta1"]), f(1 - h["beta2"])
    size = (h["lr"] / (1 - h["beta1"] ** t)).float()
    root = (1 / torch.sqrt(1 - h["beta2"] ** t)).float()
    keep, eps = f(1 - h["lr"] * h["weight_decay"]), f(h["eps"])
    eight = s["case"]["bits"] == 8
    ms, vs = [], []
    for i, (p, g) in enumerate(zip(s["p"], s["g"])):
        g = g.float()
        m = _decode(s["m"][i], s["m_scale"][i], 2, 127.0) if eight else s["m"][i]
        v = _decode(s["v"][i], s["v_scale"][i], 4, 255.0) if eight else s["v"][i]
        m = m * b1 + g * c1
        v = v * b2 + (g * g) * c2
        p.copy_(p * keep - size * (m / (torch.sqrt(v) * root + eps)))
        if s["copy"] is not None:
            s["copy"][i].copy_(p)
        if not eight:
            s["m"][i].copy_(m)
            s["v"][i].copy_(v)
            continue
        key = _pcg(_pcg(s["step"] ^ _pcg((s["seed"] & 0xFFFFFFFF) ^ _pcg(s["seed"] >> 32))) ^ i)
        r = _pcg(torch.arange(p.numel(), device=dev).view(p.shape) ^ key)
        for name, x, u, power, most in (("m", m, r & 0xFFFF, 2, 127.0), ("v", v, r >> 16, 4, 255.0)):
            code, scale = _encode(x, u, power, most)
            s[name][i].copy_(code)
            s[name + "_scale"][i].copy_(scale)
            (ms if name == "m" else vs).append(_decode(s[name][i], scale, power, most).view(-1))
    res = {"p": s["p"], "m": torch.cat(ms) if eight else s["m"], "v": torch.cat(vs) if eight else s["v"]}
    if s["copy"] is not None:
        res["copy"] = s["copy"]
    return res


# --------------------------------------------------------- the library's calls
def _dtype_code(binding, dt):
    return binding.LSTM_F32 if dt == torch.float32 else binding.LSTM_BF16


def _att_own(s):
    from layer_lstm_b200 import binding
    case = s["case"]
    if "desc" not in s:     # the description and the scratch that a program keeps
        s["desc"] = binding.make_attention_desc(case["B"], case["T"], case["H"], case["dk"], case["dv"],
                                                batch_first=case["batch_first"],
                                                dtype=_dtype_code(binding, s["q"].dtype))
        s["ws"] = torch.empty(binding.lstm_linear_attention_workspace_size(s["desc"]), device="cuda",
                              dtype=torch.uint8)
    binding.check(binding.lstm_linear_attention_forward(
        s["desc"], s["q"], s["k"], s["v"], s["log_decay"], s["s0"], s["out"], s["s_n"], s["ws"],
        lengths=s["lengths"]))
    res = {"out": s["out"], "s_n": s["s_n"]}
    if case["train"]:
        binding.check(binding.lstm_linear_attention_backward(
            s["desc"], s["q"], s["k"], s["v"], s["log_decay"], s["s0"], s["grad_out"], s["grad_sn"],
            s["dq"], s["dk"], s["dv"], s["ds0"], s["ws"], lengths=s["lengths"]))
        res.update(dq=s["dq"], dk=s["dk"], dv=s["dv"], ds0=s["ds0"])
    return res


def _step_own(s):
    from layer_lstm_b200 import binding
    case = s["case"]
    if "desc" not in s:
        s["desc"] = binding.make_attention_desc(case["B"], 1, case["H"], case["dk"], case["dv"],
                                                dtype=_dtype_code(binding, s["q"].dtype))
    binding.check(binding.lstm_linear_attention_step(s["desc"], s["q"], s["k"], s["v"], s["log_decay"],
                                                     s["state"], s["out"]))
    return {"out": s["out"], "state": s["state"]}


def _norm_own(s):
    from layer_lstm_b200 import binding
    case = s["case"]
    if "desc" not in s:
        s["desc"] = binding.make_norm_desc(case["rows"], case["cols"], dtype=_dtype_code(binding, s["x"].dtype),
                                           eps=1e-5)
        s["ws"] = torch.empty(binding.lstm_layer_norm_workspace_size(s["desc"]), device="cuda", dtype=torch.uint8)
    binding.check(binding.lstm_layer_norm_forward(s["desc"], s["x"], s["weight"], s["bias"], s["y"], s["mean"],
                                                  s["rstd"]))
    res = {"y": s["y"], "mean": s["mean"], "rstd": s["rstd"]}
    if case["train"]:
        binding.check(binding.lstm_layer_norm_backward(
            s["desc"], s["grad_y"], s["x"], s["weight"], s["mean"], s["rstd"], s["dx"], s["dweight"], s["dbias"],
            s["ws"]))
        res.update(dx=s["dx"], dweight=s["dweight"], dbias=s["dbias"])
    return res


def _adamw_own(s):
    if "opt" not in s:
        from layer_lstm_b200.optim import AdamW
        s["opt"] = AdamW(s["p"], s["g"], copies=s["copy"], state_bits=s["case"]["bits"], seed=s["seed"],
                         state=dict(m=s["m"], v=s["v"], m_scale=s.get("m_scale"), v_scale=s.get("v_scale"),
                                    step=s["step"]), **s["hyper"])
    s["opt"].step()
    res = {"p": s["p"], "m": s["m"], "v": s["v"]}
    if s["case"]["bits"] == 8:
        # the moments as float32 values, as a program takes them for a checkpoint
        s["opt"].read_state(s["m_out"], s["v_out"])
        res["m"], res["v"] = s["m_out"], s["v_out"]
    if s["copy"] is not None:
        res["copy"] = s["copy"]
    return res


def run(state):
    op = state["case"]["op"]
    if own:
        return {"att": _att_own, "att_step": _step_own, "norm": _norm_own, "adamw": _adamw_own}[op](state)
    return {"att": _att_plain, "att_step": _step_plain, "norm": _norm_plain, "adamw": _adamw_plain}[op](state)


def work(case):
    if case["op"] in ("att", "att_step"):
        e = 2 if case["dtype"] == "bf16" else 4
        heads, dk, dv = case["B"] * case["H"], case["dk"], case["dv"]
        n = heads * case.get("T", 1)
        state = heads * dk * dv * 4
        if case["op"] == "att_step":
            return {"bytes": e * n * 2 * (dk + dv) + 2 * state, "flops": 4 * n * dk * dv}
        by = e * n * 2 * (dk + dv) + state * (2 if case["s0"] else 1)
        fl = 4 * n * dk * dv
        if case["train"]:   # reads q, k, v, grad_out, s0, grad_sn again or anew; writes dq, dk, dv, ds0
            by += e * n * (2 * (dk + dv) + 2 * dk + dv) + state * (3 if case["s0"] else 2)
            fl += 10 * n * dk * dv
        return {"bytes": by, "flops": fl}
    if case["op"] == "norm":
        e = 2 if case["dtype"] == "bf16" else 4
        n, r, c = case["rows"] * case["cols"], case["rows"], case["cols"]
        by, fl = 2 * e * n + 8 * r + 2 * e * c, 8 * n
        if case["train"]:
            by, fl = by + 3 * e * n + 8 * r + e * c + 8 * c, fl + 14 * n
        return {"bytes": by, "flops": fl}
    n = sum(math.prod(z) for z in _shapes(case))
    per = 8 + (4 if case["grad"] == "f32" else 2) + (16 if case["bits"] == 32 else 4) + (2 if case["copy"] else 0)
    if case["bits"] == 8:
        per += 16 / BLOCK + 8          # scales; the moments written out as values
    return {"bytes": int(n * per), "flops": 16 * n}


# ------------------------------------------------------------------ the values
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "att_step":
        d = {a: s[a].double() for a in ("q", "k", "v", "state", "log_decay")}
        st = d["state"] * d["log_decay"].exp().view(1, -1, 1, 1)
        st = st + torch.einsum("bthi,bthj->bhij", d["k"], d["v"])
        return {"out": torch.einsum("bthi,bhij->bthj", d["q"], st) / math.sqrt(case["dk"]), "state": st}
    if case["op"] == "att":
        return _att_exact(s)
    if case["op"] == "norm":
        leaf = [s[a].double().requires_grad_() for a in ("x", "weight", "bias")]
        x, w, b = leaf
        var, mean = torch.var_mean(x, 1, correction=0)
        rstd = (var + 1e-5) ** -0.5
        y = (x - mean[:, None]) * rstd[:, None] * w + b
        res = {"y": y.detach(), "mean": mean.detach(), "rstd": rstd.detach()}
        if case["train"]:
            res.update(zip(("dx", "dweight", "dbias"), torch.autograd.grad(y, leaf, s["grad_y"].double())))
        return res
    h, t = s["hyper"], 1001
    ps, ms, vs = [], [], []
    for i, (p, g) in enumerate(zip(s["p"], s["g"])):
        m, v, p, g = s["m"][i].double(), s["v"][i].double(), p.double(), g.double()
        if case["bits"] == 8:
            a, b = (torch.repeat_interleave(s[n][i].double(), BLOCK)[: p.numel()].view(p.shape)
                    for n in ("m_scale", "v_scale"))
            m, v = m.sign() * (m / 127) ** 2 * a, (v / 255) ** 4 * b
        m, v = m.lerp(g, 1 - h["beta1"]), v.lerp(g * g, 1 - h["beta2"])
        hat = (m / (1 - h["beta1"] ** t)) / ((v / (1 - h["beta2"] ** t)).sqrt() + h["eps"])
        ps.append(p - h["lr"] * (hat + h["weight_decay"] * p))
        ms.append(m)
        vs.append(v)
    # the 8-bit moments are rounded by random numbers: no value of their own
    res = {"p": ps, "m": ms if case["bits"] == 32 else None, "v": vs if case["bits"] == 32 else None}
    if case["copy"]:
        res["copy"] = ps
    return res


def _att_exact(s):
    """The full score matrix of each batch row, a block of its rows at a time, in 64 bits; gradients by
    autograd."""
    case = s["case"]
    B, T, H, dk, dv = (case[a] for a in ("B", "T", "H", "dk", "dv"))
    bf = case["batch_first"]
    if case["train"] and H * T * T * 8 > 4e9 or B * H * T * T * (dk + dv) * 2 > 1e14:
        return None
    ld = s["log_decay"].double()
    dev = ld.device
    names = ["q", "k", "v"] + (["s0"] if s["s0"] is not None else [])
    res = {n: [] for n in ["out", "s_n"] + (["dq", "dk", "dv", "ds0"] if case["train"] else [])}
    for b in range(B):
        n = int(s["lengths"][b]) if s["lengths"] is not None else T
        row = {a: (s[a][b, :n] if bf else s[a][:n, b]).double() for a in ("q", "k", "v")}
        row["s0"] = s["s0"][b].double() if s["s0"] is not None else torch.zeros(H, dk, dv, device=dev).double()
        for x in row.values():
            x.requires_grad_(case["train"])
        at = torch.arange(n, device=dev).double()
        parts = []
        for i in range(0, n, 2048):
            far = at[i:i + 2048, None] - at[None]
            wgt = torch.where(far >= 0, torch.exp(ld.view(H, 1, 1) * far.clamp(min=0)), 0.0)
            part = torch.einsum("hij,jhv->ihv", torch.einsum("ihd,jhd->hij", row["q"][i:i + 2048], row["k"]) * wgt,
                                row["v"])
            hist = torch.exp(ld[None] * (at[i:i + 2048, None] + 1))[..., None]
            parts.append(part + hist * torch.einsum("ihd,hdv->ihv", row["q"][i:i + 2048], row["s0"]))
        out = torch.cat(parts) if parts else torch.zeros(0, H, dv, device=dev).double()
        out = out / math.sqrt(dk)
        kw = row["k"] * torch.exp(ld[None] * (n - 1 - at)[:, None])[..., None]
        s_n = torch.einsum("jhd,jhv->hdv", kw, row["v"]) + torch.exp(ld * n).view(H, 1, 1) * row["s0"]
        if case["train"]:
            go = (s["grad_out"][b, :n] if bf else s["grad_out"][:n, b]).double()
            grads = torch.autograd.grad((out * go).sum() + (s_n * s["grad_sn"][b].double()).sum(),
                                        [row[a] for a in ("q", "k", "v", "s0")], allow_unused=True,
                                        materialize_grads=True)
            for a, x in zip(("dq", "dk", "dv", "ds0"), grads):
                res[a].append(x)
        res["out"].append(out.detach())
        res["s_n"].append(s_n.detach())

    def whole(a):
        if a in ("s_n", "ds0"):
            return torch.stack(res[a])
        rows = [torch.nn.functional.pad(x, (0, 0, 0, 0, 0, T - x.shape[0])) for x in res[a]]
        return torch.stack(rows, 0 if bf else 1)

    return {a: whole(a) for a in res}

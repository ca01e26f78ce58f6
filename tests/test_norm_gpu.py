"""lstm_layer_norm_* against the equations in float64 (GPU).

Tolerances, in half-steps H = 2^-24 of float32 and half a step of the output
type.  A row's sum passes at most N = 64 + cols / 32 roundings, so the mean is
off by N H mean|x| and y by that times rstd and N H |xhat| for rstd's and the
last products, times |weight|.  The backward is given a mean and rstd that the
reference uses too: xhat is off by 3 H (|x| + |mean|) rstd, the row's means by
N H of the mean of magnitudes.  A column's sum passes at most M = 256 +
rows / 64 roundings.
"""
import pytest
import torch

from layer_lstm_b200 import binding

pytestmark = pytest.mark.gpu

H = 2.0 ** -24
SHAPES = [(1, 1), (3, 7), (1, 8192), (20, 16), (5, 17), (257, 33), (64, 100), (33, 128), (130, 250), (999, 256),
          (64, 500), (31, 512), (77, 1000), (40, 1024), (19, 2000), (37, 2048), (300, 2056), (9, 4096), (6, 5001),
          (11, 8200), (3, 20000), (5, 40000), (70001, 24), (3000, 512), (2500, 2048)]


def _make(rows, cols, dt, seed=0, offset=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def f(*shape, std=1.0, mean=0.0):
        n = 1
        for k in shape:
            n *= k
        return (torch.randn(n + offset, generator=g, device="cuda") * std + mean).to(dt)[offset:].view(*shape)

    return f(rows, cols, std=0.7, mean=0.3), f(cols, std=0.2, mean=1.0), f(cols, std=0.2), f(rows, cols)


def _out_half_step(dt):
    return torch.finfo(dt).eps / 2


def _check_forward(x, w, b, y, mean, rstd, eps):
    N = 64 + x.shape[1] / 32
    xd = x.double()
    m = xd.mean(1, keepdim=True)
    var = (xd - m).square().mean(1, keepdim=True)
    r = 1 / (var + eps).sqrt()
    xhat = (xd - m) * r
    wd = w.double() if w is not None else torch.ones(x.shape[1], device="cuda").double()
    ref = xhat * wd + (b.double() if b is not None else 0)
    ax = xd.abs().mean(1, keepdim=True)
    # the variance's own error from the mean's is of second order; the rest is relative
    tol = (N * H * ax * r + N * H * xhat.abs()) * wd.abs() + 2 * H * ref.abs() + _out_half_step(y.dtype) * ref.abs()
    assert ((y.double() - ref).abs() <= tol).all(), ((y.double() - ref).abs() / tol).max()
    if mean is not None:
        assert ((mean.double() - m[:, 0]).abs() <= N * H * ax[:, 0]).all()
        assert ((rstd.double() - r[:, 0]).abs() <= N * H * r[:, 0]).all()


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_forward(rows, cols, dt, cuda_lib):
    if cols == 1:
        eps = 1.0   # one column: y is the bias
    else:
        eps = 1e-5
    code = binding.LSTM_F32 if dt == torch.float32 else binding.LSTM_BF16
    d = binding.make_norm_desc(rows, cols, code, eps)
    for offset in (0, 1):
        x, w, b, _ = _make(rows, cols, dt, 1, offset)
        for ww, bb, stats in ((w, b, True), (None, b, False), (w, None, True)):
            y = torch.full((rows * cols + offset,), 7.0, device="cuda", dtype=dt)[offset:].view(rows, cols)
            mean, rstd = (torch.zeros(rows, device="cuda") for _ in range(2)) if stats else (None, None)
            binding.check(binding.lstm_layer_norm_forward(d, x, ww, bb, y, mean, rstd))
            _check_forward(x, ww, bb, y, mean, rstd, d.eps)


@pytest.mark.parametrize("rows,cols", SHAPES)
@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_backward(rows, cols, dt, cuda_lib):
    code = binding.LSTM_F32 if dt == torch.float32 else binding.LSTM_BF16
    d = binding.make_norm_desc(rows, cols, code, 1e-5)
    ws = torch.empty(binding.lstm_layer_norm_workspace_size(d), device="cuda", dtype=torch.uint8)
    N, M = 64 + cols / 32, 256 + rows / 64
    for offset in (0, 1):
        x, w, _, gy = _make(rows, cols, dt, 2, offset)
        mean = x.float().mean(1)
        rstd = 1 / (x.float().var(1, correction=0) + 1e-5).sqrt()
        for ww, sums in ((w, True), (None, True), (w, False)):
            dx = torch.full((rows * cols + offset,), 7.0, device="cuda", dtype=dt)[offset:].view(rows, cols)
            dw, db = (torch.full((cols,), 7.0, device="cuda") for _ in range(2)) if sums else (None, None)
            ws.fill_(255)
            binding.check(binding.lstm_layer_norm_backward(d, gy, x, ww, mean, rstd, dx, dw, db, ws if sums else None))
            r, m = rstd.double()[:, None], mean.double()[:, None]
            xhat = (x.double() - m) * r
            xe = 3 * H * (x.double().abs() + m.abs()) * r
            g = gy.double() * (ww.double() if ww is not None else 1)
            mg, mgx = g.mean(1, keepdim=True), (g * xhat).mean(1, keepdim=True)
            ref = r * (g - mg - xhat * mgx)
            me, mxe = N * H * g.abs().mean(1, keepdim=True), (N * H * (g * xhat).abs() + g.abs() * xe).mean(1, keepdim=True)
            tol = r * (4 * H * (g.abs() + mg.abs() + (xhat * mgx).abs()) + me + xhat.abs() * mxe + xe * mgx.abs())
            tol = tol * (1 + 4 * H) + _out_half_step(dt) * ref.abs() * (1 + 2.0 ** -8)
            tol = tol + _out_half_step(dt) * tol
            assert ((dx.double() - ref).abs() <= tol).all(), ((dx.double() - ref).abs() / tol).max()
            if sums:
                for got, term, err in ((dw, gy.double() * xhat, gy.double().abs() * xe), (db, gy.double(), None)):
                    bound = M * H * term.abs().sum(0) + (err.sum(0) if err is not None else 0)
                    assert ((got.double() - term.sum(0)).abs() <= bound).all()


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", [(50, 64), (50, 2048), (50, 2049)])
def test_in_place_and_alone(rows, cols, dt, cuda_lib):
    """y over x, dx over grad_y or x, dweight or dbias alone: bit for bit what separate buffers give."""
    code = binding.LSTM_F32 if dt == torch.float32 else binding.LSTM_BF16
    d = binding.make_norm_desc(rows, cols, code)
    ws = torch.empty(binding.lstm_layer_norm_workspace_size(d), device="cuda", dtype=torch.uint8)
    x, w, b, gy = _make(rows, cols, dt, 3)
    y, mean, rstd = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    binding.check(binding.lstm_layer_norm_forward(d, x, w, b, y, mean, rstd))
    z = x.clone()
    binding.check(binding.lstm_layer_norm_forward(d, z, w, b, z))
    assert torch.equal(z, y)
    dx, dw, db = torch.empty_like(x), torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    binding.check(binding.lstm_layer_norm_backward(d, gy, x, w, mean, rstd, dx, dw, db, ws))
    for over in ("gy", "x"):
        t = dict(gy=gy.clone(), x=x.clone())
        dw2, db2 = torch.empty_like(dw), torch.empty_like(db)
        binding.check(binding.lstm_layer_norm_backward(d, t["gy"], t["x"], w, mean, rstd, t[over], dw2, db2, ws))
        assert torch.equal(t[over], dx) and torch.equal(dw2, dw) and torch.equal(db2, db)
    for want in ("dw", "db"):
        o = torch.empty(cols, device="cuda")
        binding.check(binding.lstm_layer_norm_backward(d, gy, x, w, mean, rstd, None, o if want == "dw" else None,
                                                       o if want == "db" else None, ws))
        assert torch.equal(o, dw if want == "dw" else db)


def test_no_rows(cuda_lib):
    d = binding.make_norm_desc(0, 10)
    ws = torch.empty(binding.lstm_layer_norm_workspace_size(d), device="cuda", dtype=torch.uint8)
    dw, db = torch.ones(10, device="cuda"), torch.ones(10, device="cuda")
    binding.check(binding.lstm_layer_norm_backward(d, None, None, None, None, None, None, dw, db, ws))
    assert (dw == 0).all() and (db == 0).all()


def test_rows_do_not_mix(cuda_lib):
    """A row with a NaN or an infinity leaves the other rows as they are; a constant row gives the bias."""
    d = binding.make_norm_desc(6, 300)
    x, w, b, _ = _make(6, 300, torch.float32, 4)
    x[1, 7], x[3, 9] = float("nan"), float("inf")
    x[5] = 3.25
    y = torch.empty_like(x)
    binding.check(binding.lstm_layer_norm_forward(d, x, w, b, y))
    assert y[1].isnan().all() and y[3].isnan().any() and y[[0, 2, 4, 5]].isfinite().all()
    assert torch.equal(y[5], b)


@pytest.mark.parametrize("dt", [torch.float32, torch.bfloat16])
def test_against_differences(dt, cuda_lib):
    """The gradients against autograd of the equations in float64 and, in float32, central differences of the
    library's own forward along one direction (step 1e-2; its curvature and the forward's rounding leave 1e-3)."""
    rows, cols = 40, 200
    code = binding.LSTM_F32 if dt == torch.float32 else binding.LSTM_BF16
    d = binding.make_norm_desc(rows, cols, code)
    ws = torch.empty(binding.lstm_layer_norm_workspace_size(d), device="cuda", dtype=torch.uint8)
    x, w, b, gy = _make(rows, cols, dt, 5)
    y, mean, rstd = torch.empty_like(x), torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    binding.check(binding.lstm_layer_norm_forward(d, x, w, b, y, mean, rstd))
    dx, dw, db = torch.empty_like(x), torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
    binding.check(binding.lstm_layer_norm_backward(d, gy, x, w, mean, rstd, dx, dw, db, ws))
    leaf = [t.double().requires_grad_() for t in (x, w, b)]
    ref = torch.nn.functional.layer_norm(leaf[0], (cols,), leaf[1], leaf[2], d.eps)
    for got, want in zip((dx, dw, db), torch.autograd.grad(ref, leaf, gy.double())):
        # 2^-8 bf16 rounding of dx; float32 sums otherwise
        bound = 2 * _out_half_step(dt) if got is dx else 1e-5
        assert (got.double() - want).norm() <= max(bound, 1e-5) * want.norm()
    if dt == torch.float32:
        u = torch.randn_like(x)
        vals = []
        for sgn in (1, -1):
            y2 = torch.empty_like(x)
            binding.check(binding.lstm_layer_norm_forward(d, x + sgn * 1e-2 * u, w, b, y2))
            vals.append((y2.double() * gy.double()).sum().item())
        want = (dx.double() * u.double()).sum().item()
        assert abs((vals[0] - vals[1]) / 2e-2 - want) <= 1e-3 * (dx.double() * u.double()).abs().sum().item()


def test_captured_calls_share_a_workspace(cuda_lib):
    """Two captured backward passes over one workspace, replayed in turn on one stream."""
    rows, cols = 700, 96
    d = binding.make_norm_desc(rows, cols)
    ws = torch.empty(binding.lstm_layer_norm_workspace_size(d), device="cuda", dtype=torch.uint8)
    s = torch.cuda.Stream()
    sets, graphs = [], []
    for seed in (6, 7):
        x, w, b, gy = _make(rows, cols, torch.float32, seed)
        t = dict(x=x, w=w, b=b, gy=gy, y=torch.empty_like(x), mean=torch.empty(rows, device="cuda"),
                 rstd=torch.empty(rows, device="cuda"), dx=torch.empty_like(x), dw=torch.empty(cols, device="cuda"),
                 db=torch.empty(cols, device="cuda"))

        def call(stream=None, t=t):
            binding.check(binding.lstm_layer_norm_forward(d, t["x"], t["w"], t["b"], t["y"], t["mean"], t["rstd"], stream))
            binding.check(binding.lstm_layer_norm_backward(d, t["gy"], t["x"], t["w"], t["mean"], t["rstd"], t["dx"],
                                                           t["dw"], t["db"], ws, stream))
        call()
        torch.cuda.synchronize()
        sets.append((t, {k: t[k].clone() for k in ("y", "dx", "dw", "db")}))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call(s)
        graphs.append(g)
    for t, _ in sets:
        for k in ("y", "dx", "dw", "db"):
            t[k].zero_()
    for _ in range(2):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for t, want in sets:
        for k, v in want.items():
            assert torch.equal(t[k], v), k

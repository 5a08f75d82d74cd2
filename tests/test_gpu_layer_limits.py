"""The layer-side operators where their sums are long, their gates extreme and their launches many turns
long, against fp64 on the GPU.  Bounds as in test_gpu_layer: u = 2^-24, a bf16 result lies between the bf16
roundings of the two ends of its interval."""
import numpy as np
import pytest

from oracle import layer_ref as L
from test_gpu_layer import U, close, dt, f64, filled, held, mu, plan, rand, values  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ weight gradient
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("expert", [True, False])
@pytest.mark.parametrize("n", [32, 31])
def test_wgrad_of_many_tokens_does_not_drift(mu, plan, dtype, expert, n):
    """2^21 tokens of one sign.  The gradient starts at minus the sum, rounded, so that what is left shows
    the sum's own error.  At most 2048 tokens per accumulator of the tensor cores, whose adds truncate (2 u
    per token), then fp32 sums of those: u per partial sum."""
    import torch
    t, m = 1 << 21, 16
    gen = torch.Generator(device="cuda").manual_seed(1)
    dy = (0.5 + 0.5 * torch.rand((t, m), generator=gen, device="cuda")).bfloat16()
    x8 = filled(mu, 0.5 + 0.5 * torch.rand((t, n), generator=gen, device="cuda"), "int8")
    x = torch.empty((t, n), device="cuda")
    mu.act_unpack(x8, x)
    want = torch.zeros((m, n), dtype=torch.float64, device="cuda")
    for a in range(0, t, t // 8):
        want += dy[a:a + t // 8].double().t() @ x[a:a + t // 8].double()
    g = (-want).to(dt(dtype))
    g0 = f64(g)
    if expert:
        plan.wgrad(dy, x8, g.unsqueeze(0), offsets=torch.tensor([0, t], dtype=torch.int32, device="cuda"), accumulate=True)
    else:
        plan.wgrad(dy, x8, g, accumulate=True)
    plan.sync()
    want = want.cpu().numpy()
    close(g, want + g0, (2 * (2048 + 8) + t // 2048 + 4) * U * want)


def close_gpu(got, want, bound):
    """``close`` for tensors of the GPU without NaN; fp64 ``want`` and ``bound``."""
    import torch
    if got.dtype is torch.bfloat16:   # torch rounds fp64 to bf16 by way of fp32: one fp32 step outwards covers that
        lo, hi = ((want + s * (bound + 2 * U * want.abs())).bfloat16() for s in (-1, 1))
        assert bool(((lo <= got) & (got <= hi)).all())
    else:
        assert bool(((got.double() - want).abs() <= bound).all())


def unpacked(mu, a):
    import torch
    y = torch.empty((a.rows, a.cols), device="cuda")
    mu.act_unpack(a, y)
    return y.double()


@pytest.mark.parametrize("m,n", [(2312, 2308), (2311, 2304)])
@pytest.mark.parametrize("dtype,accumulate,scaled", [("bf16", False, True), ("f32", True, False), ("bf16", True, False),
                                                     ("f32", False, True)])
def test_wgrad_of_more_tiles_than_pairs(mu, plan, m, n, dtype, accumulate, scaled):
    """Two bands of tiles along m, the second narrower; whole tiles first, the last turn's split along the tokens."""
    import torch
    t = 8200
    dy, x8 = rand((t, m), "bf16", 1, 0.5), filled(mu, rand((t, n), "f32", 2, 2.0), "e4m3")
    s = 1 + 0.3 * rand((1, n), "f32", 3)[0] if scaled else torch.ones(n, device="cuda")
    g = rand((m, n), dtype, 4).contiguous()
    g0 = g.double() if accumulate else torch.zeros((), dtype=torch.float64, device="cuda")
    d, x = dy.double(), unpacked(mu, x8)
    want = d.t() @ x * s.double() + g0
    bound = 2 * (t + 8) * U * (d.abs().t() @ x.abs()) * s.double().abs() + 4 * U * (want.abs() + g0.abs()) + 1e-30
    plan.wgrad(dy, x8, g, col_scale=s if scaled else None, accumulate=accumulate)
    plan.sync()
    close_gpu(g, want, bound)


# ------------------------------------------------------------------ SwiGLU
def silu_bound(g, u):
    """|error| of silu(g) u: the exponential 2 ulp and its correction's rounding (5 u), 1 + e (u), the reciprocal
    2^-23 on [1, 2) (4 u), two products (2 u)."""
    return 12 * U * (g * L.sigmoid(g) * u).__abs__()


def test_silu_over_all_gates(mu):
    """Gates evenly over [-87, 87], so the sigmoid from 1.6e-38 to 1."""
    import torch
    g = torch.linspace(-87, 87, 64 * 1024, device="cuda").view(64, 1024)
    u = torch.ones_like(g)
    a = torch.empty_like(g)
    mu.swiglu_forward(g, u, a)
    close(a, L.swiglu(f64(g), f64(u)), silu_bound(f64(g), f64(u)))


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_silu_gradient_over_all_gates(mu, fmt):
    import torch
    g = torch.linspace(-87, 87, 64 * 1024, device="cuda").view(64, 1024)
    u, d = rand((64, 1024), "f32", 1), rand((64, 1024), "f32", 2)
    g8, u8, dg, du = filled(mu, g, fmt), filled(mu, u, fmt), torch.empty_like(d), torch.empty_like(d)
    mu.swiglu_backward(d, g8, u8, dg, du)
    g, u, d = values(g8), values(u8), f64(d)
    s = L.sigmoid(g)
    wg, wu = L.swiglu_grad(d, g, u)
    # s (10 u), silu (11 u), 1 - s (10 u of s), their product, sum and the two products with da and up
    close(dg, wg, 16 * U * np.abs(d * u) * s * np.where(g < 0, 1 - g * (1 - s), 1 + g) + 1e-44)
    close(du, wu, 12 * U * np.abs(wu) + 1e-44)


def test_silu_of_gates_that_are_not_finite(mu):
    import torch
    inf, nan = float("inf"), float("nan")
    g = torch.tensor([[inf, -inf, nan, 0.0, 1.0, 2.0, -200.0, 200.0]], device="cuda")
    u = torch.tensor([[2.0, 2.0, 2.0, inf, inf, nan, 2.0, 2.0]], device="cuda")
    with np.errstate(all="ignore"):
        want = f64(g) / (1 + np.exp(-f64(g))) * f64(u)
    for dtype in ("f32", "bf16"):
        a, g8 = torch.empty_like(g, dtype=dt(dtype)), mu.Act8.empty(1, 8)
        mu.swiglu_forward(g.to(dt(dtype)), u.to(dt(dtype)), a, saved_gate=g8)
        close(a.float(), want, np.full(8, 1e-30))
        d, dg, du = torch.ones_like(a), torch.empty_like(a), torch.empty_like(a)
        mu.swiglu_backward(d, g8, filled(mu, torch.ones_like(u), "e4m3"), dg, du)
        assert dg.isnan().all() and du.isnan().all()     # the group of eight reads back as NaN


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("cols,pad", [(640, 0), (641, 0), (513, 3)])
def test_swiglu_forward_in_place(mu, dtype, cols, pad):
    import torch
    g, u = rand((40, cols), dtype, 1, 2.0, pad), rand((40, cols), dtype, 2, 2.0, pad)
    a = torch.empty((40, cols), dtype=dt(dtype), device="cuda")
    mu.swiglu_forward(g, u, a)
    g0, u0 = g.clone(), u.clone()
    mu.swiglu_forward(g, u0, g)
    mu.swiglu_forward(g0, u, u)
    assert torch.equal(g, a) and torch.equal(u, a)


# ------------------------------------------------------------------ launches of many turns
MANY = [(9000, 2600, 0), (9000, 2601, 0), (40000, 600, 0), (40000, 599, 3), (90000, 100, 0)]


@pytest.mark.parametrize("rows,cols,pad", MANY)
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_packing_in_many_turns(mu, rows, cols, pad, fmt):
    """More units than launched warps: the codes of calls of a few rows each, and their values."""
    import torch
    x = rand((rows, cols), "bf16", 1, 3.0, pad)
    whole = filled(mu, x, fmt)
    part = mu.Act8.empty(rows, cols, fmt)
    for r in range(0, rows, 1000):
        mu.act_pack(x[r:r + 1000], mu.Act8(part.codes[r:r + 1000], part.scales[r:r + 1000], cols, fmt))
    groups = (cols + 31) // 32
    assert torch.equal(whole.codes[:, :cols], part.codes[:, :cols])
    assert torch.equal(whole.scales[:, :groups], part.scales[:, :groups])
    for r in (0, rows // 2, rows - 1):
        assert np.array_equal(held(whole)[0][r:r + 1], L.pack(f64(x[r:r + 1]), fmt)[0])
    y = unpacked(mu, whole)
    step = torch.exp2(whole.scales[:, :groups].double() - 127).repeat_interleave(32, 1)[:, :cols]
    half = 0.5 * step if fmt == "int8" else torch.maximum(x.double().abs() / 16, 2.0 ** -10 * step)
    assert bool(((y - x.double()).abs() <= half).all())
    wide = torch.empty((rows, cols + 2 * pad), dtype=torch.bfloat16, device="cuda")
    out = wide[:, pad:pad + cols]
    mu.act_unpack(whole, out)
    assert torch.equal(out.double(), y)


@pytest.mark.parametrize("rows,cols,pad", MANY)
def test_swiglu_in_many_turns(mu, rows, cols, pad):
    import torch
    g, u, d = (rand((rows, cols), "bf16", k, s, pad) for k, s in ((1, 3.0), (2, 1.0), (3, 0.1)))
    a, g8, u8 = torch.empty_like(g), mu.Act8.empty(rows, cols), mu.Act8.empty(rows, cols)
    mu.swiglu_forward(g, u, a, saved_gate=g8, saved_up=u8)
    G, V, D = g.double(), u.double(), d.double()
    s = torch.sigmoid(G)
    close_gpu(a, G * s * V, 12 * U * (G * s * V).abs() + 1e-30)
    for x, q in ((g, g8), (u, u8)):
        p = filled(mu, x, "e4m3")
        groups = (cols + 31) // 32
        assert torch.equal(q.codes[:, :cols], p.codes[:, :cols]) and torch.equal(q.scales[:, :groups], p.scales[:, :groups])
    dgu, a8 = torch.empty((rows, 2 * cols), dtype=torch.bfloat16, device="cuda"), mu.Act8.empty(rows, cols)
    mu.swiglu_backward(d, g8, u8, dgu[:, :cols], dgu[:, cols:], saved_out=a8)
    G, V = unpacked(mu, g8), unpacked(mu, u8)
    s = torch.sigmoid(G)
    close_gpu(dgu[:, :cols], D * V * s * (1 + G * (1 - s)), 16 * U * (D * V).abs() * s * (1 + G.abs()) + 1e-30)
    close_gpu(dgu[:, cols:], D * G * s, 16 * U * (D * G).abs() * s + 1e-30)
    v = G * s * V
    step = torch.exp2(a8.scales[:, :(cols + 31) // 32].double() - 127).repeat_interleave(32, 1)[:, :cols]
    half = torch.maximum(v.abs() / 16, 2.0 ** -10 * step)
    assert bool(((unpacked(mu, a8) - v).abs() <= 1.001 * half + 32 * U * v.abs()).all())


@pytest.mark.parametrize("rows,cols,dtype,pad,source", [
    (6000, 1024, "bf16", 0, "int8"), (6000, 1023, "bf16", 1, "int8"), (6000, 1024, "bf16", 0, "h"),
    (1000, 16383, "bf16", 0, "int8"), (1000, 16384, "bf16", 0, "e4m3"), (1500, 8200, "f32", 0, "h"),
    (1500, 8201, "f32", 3, "int8"), (20000, 96, "bf16", 0, "e4m3"), (20000, 97, "f32", 0, "h"), (900, 32768, "f32", 0, "h"),
    (3000, 3584, "bf16", 0, "int8"), (1300, 5000, "bf16", 4, "int8")])
@pytest.mark.parametrize("in_place", [True, False])
def test_norm_backward_in_many_turns(mu, plan, rows, cols, dtype, pad, source, in_place):
    """Many rows per block: ring slots used over and over, and dx written over dy while later rows are fetched."""
    import torch
    h = rand((rows, cols), dtype, 1, 2.0, pad)
    rstd = torch.rsqrt(h.float().square().mean(1) + 1e-6)
    dy, dres = rand((rows, cols), dtype, 8, 0.1, pad), rand((rows, cols), dtype, 9, 0.1, pad)
    w = 1 + 0.3 * rand((1, cols), "f32", 3)[0]
    r = rstd.double()[:, None]
    saved = None if source == "h" else filled(mu, h.float() * rstd[:, None], source)
    n = h.double() * r if source == "h" else unpacked(mu, saved)
    D, R, W = dy.double(), dres.double(), w.double()
    t = D * W
    want = r * (t - n * (t * n).mean(1, keepdim=True)) + R
    mean = (t * n).abs().mean(1, keepdim=True)
    bound = U * (r * (6 * t.abs() + n.abs() * 106 * mean) + 2 * R.abs() + 2 * want.abs()) + 1e-30
    dw64, dwb = (D * n).sum(0), U * (rows + 20) * (D * n).abs().sum(0) + 1e-30
    dx, dw = dy if in_place else torch.empty_like(dy), torch.empty(cols, device="cuda")
    plan.rmsnorm_backward(dy, w, rstd, dx, dw, saved=saved, h=h if source == "h" else None, dres=dres)
    plan.sync()
    close_gpu(dx, want, bound)
    close_gpu(dw, dw64, dwb)


@pytest.mark.parametrize("rows,cols", [(4000, 640), (300, 3584), (50, 32767)])
def test_rstd_is_rounded_once(mu, rows, cols):
    """Rows of whole numbers, whose sums of squares fp32 holds exactly: 1 / sqrt(mean + eps) to half an ulp, and
    2^-10 of one for what the second float of the mean and the Newton step's square leave."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(3)
    top = int((2.0 ** 24 / cols) ** 0.5)
    x = torch.randint(-min(top, 20), min(top, 20) + 1, (rows, cols), generator=gen, device="cuda").float()
    eps, rstd = 2.0 ** -20, torch.empty(rows, device="cuda")
    mu.rmsnorm_forward(x, torch.ones(cols, device="cuda"), eps, rstd=rstd)
    want = 1 / np.sqrt(np.sum(f64(x) ** 2, 1) / cols + eps)
    ulp = np.spacing(want.astype(np.float32)).astype(np.float64)
    assert np.max(np.abs(f64(rstd) - want) / ulp) <= 0.5 + 2.0 ** -10


# ------------------------------------------------------------------ rows of an Act8 inside a longer buffer
@pytest.mark.parametrize("cols", [1001, 1007, 9, 33])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_writers_keep_to_the_row(mu, cols, dtype):
    """Codes and scales that are views into a longer buffer: what lies beside them stays as it was."""
    import torch
    x = rand((1, cols), dtype, 1, 2.0)
    groups = (cols + 31) // 32

    def view():
        buf = torch.full((2, 4096), 0xA5, dtype=torch.uint8, device="cuda")
        return buf, mu.Act8(buf[:1, :cols], buf[1:, :groups], cols, "int8")

    def check(buf, want):
        assert torch.equal(buf[0, :cols], want.codes[0, :cols]) and torch.equal(buf[1, :groups], want.scales[0, :groups])
        assert bool((buf[0, cols:] == 0xA5).all()) and bool((buf[1, groups:] == 0xA5).all())

    want = filled(mu, x, "int8")
    buf, a = view()
    mu.act_pack(x, a)
    check(buf, want)
    buf, a = view()
    mu.swiglu_forward(x, x, saved_gate=a)
    check(buf, want)
    buf, a = view()
    w, y = torch.ones(cols, device="cuda"), mu.Act8.empty(1, cols, "int8")
    mu.rmsnorm_forward(x, w, 1e-6, saved=y)
    mu.rmsnorm_forward(x, w, 1e-6, saved=a)
    check(buf, y)
    buf, a = view()
    d, dg, du = torch.ones_like(x), torch.empty_like(x), torch.empty_like(x)
    mu.swiglu_backward(d, want, want, dg, du, saved_out=y)
    mu.swiglu_backward(d, want, want, dg, du, saved_out=a)
    check(buf, y)

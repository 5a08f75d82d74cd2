"""The layer-side operators on the GPU against their fp64 definitions (oracle/layer_ref.py).

Bounds, with u = 2^-24 (fp32 unit roundoff): packing and unpacking are exact, so codes and
scales have to be equal; sums of K terms carry (K + small) u of the terms' magnitudes
(twice that where the tensor cores' truncating adds form them).  A bf16 output has to lie
between the bf16 roundings of the two ends of that interval: its own rounding needs no
tolerance."""
import numpy as np
import pytest

from oracle import layer_ref as L

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def mu():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import matrix_orthogonalising_optimizer_muon_gb300 as mu
    return mu


@pytest.fixture(scope="module")
def plan(mu):
    with mu.GradPlan() as p:
        yield p
        p.sync()


def dt(name):
    import torch
    return torch.bfloat16 if name == "bf16" else torch.float32


def rand(shape, dtype, seed, scale=1.0, pad=0):
    """A CUDA tensor of N(0, scale^2) values; pad > 0: a column block of a wider tensor, off alignment."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows, cols = shape
    w = (torch.randn((rows, cols + 2 * pad), generator=g, device="cuda") * scale).to(dt(dtype))
    return w[:, pad:pad + cols]


def f64(t):
    return t.double().cpu().numpy()


def held(a):
    """(codes, scales) of an Act8 without the padding."""
    return a.codes[:, :a.cols].cpu().numpy(), a.scales[:, :(a.cols + 31) // 32].cpu().numpy()


def values(a):
    return L.unpack(*held(a), a.fmt)


def filled(mu, x, fmt):
    a = mu.Act8.empty(x.shape[0], x.shape[1], fmt)
    mu.act_pack(x, a)
    return a


def to_bf16(x):
    """Round to nearest even to 8 significant bits (normal range)."""
    f, e = np.frexp(x)
    return np.where(np.isfinite(x), np.ldexp(np.rint(f * 256) / 256, e), x)


def close(got, want, bound):
    """want - bound <= got <= want + bound elementwise, the ends rounded to bf16 for a bf16 result; NaN where NaN is due."""
    half = str(got.dtype) == "torch.bfloat16"
    got = f64(got)
    if half:
        fine = np.isfinite(want)
        lo, hi = to_bf16(want - bound), to_bf16(want + bound)
        assert np.array_equal(np.isfinite(got), fine)
        assert np.all((lo <= got) & (got <= hi) | ~fine), np.max(np.abs(got - want)[fine])
        return
    assert np.array_equal(np.isnan(got), np.isnan(want))
    off = np.abs(got - want) - bound
    assert np.nanmax(np.where(np.isfinite(want), off, -1), initial=-1) <= 0, (np.nanmax(off), np.nanmax(np.abs(got - want)))
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf])


# ------------------------------------------------------------------ 8 bits
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,cols,pad", [(1, 1, 0), (3, 31, 0), (2, 33, 0), (5, 256, 0), (7, 257, 0), (4, 1000, 8),
                                           (130, 1001, 3), (1, 20000, 0)])
def test_pack_and_unpack_are_exact(mu, fmt, dtype, rows, cols, pad):
    import torch
    x = rand((rows, cols), dtype, rows * 1000 + cols, 3.0, pad)
    x[0, 0] = 0.0
    if cols > 40:
        x[-1, 32:64] = 0                      # a group of zeros
    a = filled(mu, x, fmt)
    q, s = L.pack(f64(x), fmt)
    gq, gs = held(a)
    assert np.array_equal(gs, s)
    assert np.array_equal(gq, q)
    for out in ("bf16", "f32"):
        y = torch.empty((rows, cols + 2 * pad), dtype=dt(out), device="cuda")[:, pad:pad + cols]
        mu.act_unpack(a, y)
        assert np.array_equal(f64(y), L.unpack(q, s, fmt))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("offset", range(8))
@pytest.mark.parametrize("pitch", [1, 4, 7, 8])
def test_rows_at_every_offset(mu, dtype, offset, pitch):
    """Rows that begin anywhere within 16 bytes: the same codes and values as aligned rows, nothing beside them touched."""
    import torch
    rows = 6
    for cols in (1, 7, 8, 9, 31, 250, 255, 256, 257, 263, 505, 511, 512, 513, 1021):
        ld = -(-cols // 8) * 8 + pitch
        wide = rand((rows + 1, ld), dtype, 100 + cols)
        flat = wide.flatten()
        x = flat[offset:offset + rows * ld].view(rows, ld)[:, :cols]
        whole = torch.zeros(rows, -(-cols // 8) * 8, dtype=dt(dtype), device="cuda")
        whole[:, :cols] = x
        got, want = mu.Act8.empty(rows, cols, "e4m3"), mu.Act8.empty(rows, cols, "e4m3")
        mu.act_pack(x, got)
        mu.act_pack(whole[:, :cols], want)
        assert all(np.array_equal(g, w) for g, w in zip(held(got), held(want)))
        expect = torch.full_like(flat, 77.0)
        y = expect.clone()
        mu.act_unpack(want, whole[:, :cols])
        expect[offset:offset + rows * ld].view(rows, ld)[:, :cols] = whole[:, :cols]
        mu.act_unpack(want, y[offset:offset + rows * ld].view(rows, ld)[:, :cols])
        assert torch.equal(y, expect)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("aligned", [True, False])
def test_pack_over_the_whole_range(mu, fmt, aligned):
    """Every bf16 pattern, infinities, NaN and subnormals among them, and magnitudes at the range's ends."""
    import torch
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).float().reshape(128, 512)
    mixed = bits.t().contiguous().reshape(128, 512)          # groups of one exponent, and groups of many
    x = torch.cat([bits, mixed]).cuda()
    wide = torch.zeros((256, 513), device="cuda")
    src = x if aligned else wide[:, 1:].copy_(x)
    a = filled(mu, src, fmt)
    q, s = L.pack(f64(x), fmt)
    gq, gs = held(a)
    assert np.array_equal(gs, s)
    ok = np.repeat(s, 32, 1) != 255
    assert np.array_equal(L.unpack(gq, gs, fmt)[ok], L.unpack(q, s, fmt)[ok])
    y = torch.empty((256, 512), dtype=torch.float32, device="cuda")
    mu.act_unpack(a, y)
    want = L.unpack(gq, gs, fmt)
    assert np.array_equal(np.isnan(f64(y)), np.isnan(want)) and np.array_equal(f64(y)[ok], want[ok])


def test_no_rows(mu, plan):
    import torch
    x = torch.empty((0, 70), device="cuda")
    a = mu.Act8.empty(0, 70)
    mu.act_pack(x, a)
    mu.act_unpack(a, x)
    w = torch.ones(70, device="cuda")
    mu.rmsnorm_forward(x, w, 1e-6, y=torch.empty_like(x))
    mu.swiglu_forward(x, x, torch.empty_like(x))
    for acc, want in ((False, 0.0), (True, 1.0)):
        dw = torch.ones(70, device="cuda")
        plan.rmsnorm_backward(x, w, torch.empty(0, device="cuda"), torch.empty_like(x), dw, saved=a, accumulate=acc)
        g = torch.ones((40, 70), device="cuda")
        plan.wgrad(torch.empty((0, 40), dtype=torch.bfloat16, device="cuda"), a, g, accumulate=acc)
        plan.sync()
        assert (dw == want).all() and (g == want).all()


# ------------------------------------------------------------------ norm
NORM = [(1, 1, "f32", 0), (3, 31, "f32", 0), (2, 256, "bf16", 0), (9, 1001, "bf16", 0), (5, 1001, "f32", 1),
        (33, 3584, "bf16", 0), (4, 3584, "bf16", 5), (3, 4104, "f32", 0), (2, 8192, "bf16", 0), (2, 12301, "f32", 0),
        (2, 32768, "bf16", 0), (700, 96, "bf16", 0)]


@pytest.mark.parametrize("rows,cols,dtype,pad", NORM)
@pytest.mark.parametrize("residual", [True, False])
def test_rmsnorm_forward(mu, rows, cols, dtype, pad, residual):
    import torch
    x, r = rand((rows, cols), dtype, 1, 2.0, pad), rand((rows, cols), dtype, 2, 1.0, pad)
    if rows > 2:
        x[1], r[1] = 0, 0                    # a padding token
    w = 1 + 0.3 * rand((1, cols), "f32", 3)[0]
    h, y = torch.empty((rows, cols), dtype=dt(dtype), device="cuda"), torch.empty((rows, cols), dtype=dt(dtype), device="cuda")
    rstd = torch.empty(rows, device="cuda")
    a = mu.Act8.empty(rows, cols, "int8")
    mu.rmsnorm_forward(x, w, 1e-6, residual=r if residual else None, h=h, y=y, saved=a, rstd=rstd)
    h64, y64, n64, r64 = L.rmsnorm(f64(x), f64(w), 1e-6, f64(r) if residual else None)
    close(h, h64, U * np.abs(h64) * 1.01)
    # sum of squares: at most 8 * 8 + 5 + 16 adds in a chain; the square root halves it
    chain = 60 * U
    close(rstd, r64, chain * r64)
    size = np.abs(y64)
    close(y, y64, (chain + 8 * U) * size * 1.01 + U * np.abs(f64(w)))
    # the 8-bit norm: half a code step of the value, plus what fp32 moved
    q, s = L.pack(n64, "int8")
    step = np.repeat(np.exp2(s.astype(np.float64) - 127), 32, 1)[:, :cols]
    assert np.max(np.abs(values(a) - n64) - (step * 0.5 + (chain + 8 * U) * (np.abs(n64) + 128 * step))) <= 0


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("cols,pad", [(3584, 0), (1001, 0), (515, 1)])
def test_rmsnorm_saved_is_the_packed_norm(mu, fmt, cols, pad):
    """With an fp32 y the saved copy is y's, code for code; with a weight of one, also unweighted."""
    import torch
    x, w = rand((17, cols), "f32", 4, 2.0, pad), 1 + 0.3 * rand((1, cols), "f32", 5)[0]
    for weight, weighted in ((w, True), (torch.ones(cols, device="cuda"), False)):
        y, a = torch.empty((17, cols), device="cuda"), mu.Act8.empty(17, cols, fmt)
        mu.rmsnorm_forward(x, weight, 1e-5, y=y, saved=a, saved_weighted=weighted)
        q, s = L.pack(f64(y), fmt)
        assert np.array_equal(held(a)[1], s) and np.array_equal(held(a)[0], q)


def test_rmsnorm_in_place_and_not_finite(mu):
    import torch
    x, r, w = rand((6, 640), "bf16", 6), rand((6, 640), "bf16", 7), torch.ones(640, device="cuda")
    h, y = torch.empty_like(x), torch.empty_like(x)
    mu.rmsnorm_forward(x, w, 1e-6, residual=r, h=h, y=y)
    x2, r2 = x.clone(), r.clone()
    mu.rmsnorm_forward(x2, w, 1e-6, residual=r2, h=r2, y=x2)
    assert torch.equal(r2, h) and torch.equal(x2, y)
    x[3, 5] = float("nan")
    a = mu.Act8.empty(6, 640)
    mu.rmsnorm_forward(x, w, 1e-6, residual=r, y=y, saved=a)
    v = values(a)
    assert np.isnan(v[3]).all() and np.isfinite(np.delete(v, 3, 0)).all() and y[3].isnan().all()


@pytest.mark.parametrize("rows,cols,dtype,pad", NORM)
@pytest.mark.parametrize("source", ["e4m3", "int8", "h"])
def test_rmsnorm_backward(mu, plan, rows, cols, dtype, pad, source):
    import torch
    h = rand((rows, cols), dtype, 1, 2.0, pad)
    rstd = torch.rsqrt(h.float().square().mean(1) + 1e-6)
    dy, dres = rand((rows, cols), dtype, 8, 0.1, pad), rand((rows, cols), dtype, 9, 0.1, pad)
    w = 1 + 0.3 * rand((1, cols), "f32", 3)[0]
    if source == "h":
        saved, n = None, f64(h) * f64(rstd)[:, None]
    else:
        saved = filled(mu, h.float() * rstd[:, None], source)
        n = values(saved)
    dx, dw = torch.empty((rows, cols), dtype=dt(dtype), device="cuda"), rand((1, cols), "f32", 10)[0].contiguous()
    dw0 = f64(dw)
    plan.rmsnorm_backward(dy, w, rstd, dx, dw, saved=saved, h=h if source == "h" else None, dres=dres, accumulate=True)
    plan.sync()
    dy64, w64, r64 = f64(dy), f64(w), f64(rstd)[:, None]
    want, dw64 = L.rmsnorm_grad(dy64, n, f64(rstd), w64, f64(dres))
    t = np.abs(dy64 * w64)
    mean = np.mean(t * np.abs(n), 1, keepdims=True)
    bound = U * (r64 * (6 * t + np.abs(n) * 100 * mean + 6 * np.abs(n) * mean) + 2 * np.abs(f64(dres)) + 2 * np.abs(want))
    close(dx, want, bound + 1e-30)
    close(dw, dw0 + dw64, U * ((rows + 20) * np.sum(np.abs(dy64 * n), 0) + 2 * np.abs(dw0)) + 1e-30)


def test_rmsnorm_backward_parts_alone_and_in_place(mu, plan):
    import torch
    h, w = rand((300, 1024), "bf16", 1, 2.0), 1 + 0.3 * rand((1, 1024), "f32", 3)[0]
    rstd, dy = torch.rsqrt(h.float().square().mean(1) + 1e-6), rand((300, 1024), "bf16", 8)
    a = filled(mu, h.float() * rstd[:, None], "int8")
    dx, dw = torch.empty_like(dy), torch.empty(1024, device="cuda")
    plan.rmsnorm_backward(dy, w, rstd, dx, dw, saved=a)
    dx1, dw1, dy1 = torch.empty_like(dy), torch.empty_like(dw), dy.clone()
    plan.rmsnorm_backward(dy, w, rstd, dx1, saved=a)
    plan.rmsnorm_backward(dy, w, rstd, dweight=dw1, saved=a)
    plan.rmsnorm_backward(dy1, w, rstd, dy1, saved=a)
    plan.sync()
    assert torch.equal(dx, dx1) and torch.equal(dw, dw1) and torch.equal(dx, dy1)


def test_rmsnorm_gradient_against_differences(mu, plan):
    """The kernels' own slope: the loss sum(y dy), forward kernel, moved along a direction, in fp32."""
    import torch
    x, w, dy, d = (rand((4, 256), "f32", k) for k in (1, 2, 3, 4))
    w = w[0].contiguous()
    y, rstd = torch.empty_like(x), torch.empty(4, device="cuda")
    mu.rmsnorm_forward(x, w, 1e-6, y=y, rstd=rstd)
    dx = torch.empty_like(x)
    plan.rmsnorm_backward(dy, w, rstd, dx, h=x)
    plan.sync()

    def loss(z):
        mu.rmsnorm_forward(z, w, 1e-6, y=y)
        return float((y.double() * dy.double()).sum())
    step = 2.0 ** -7
    slope, want = (loss(x + step * d) - loss(x - step * d)) / (2 * step), float((dx.double() * d.double()).sum())
    # second-order remainder of the central difference and fp32 rounding of y over the step
    assert abs(slope - want) <= 1e-3 * float((dx.double() * d.double()).abs().sum())


# ------------------------------------------------------------------ SwiGLU
GLU = [(1, 1, "f32", 0), (2, 33, "bf16", 0), (5, 1000, "bf16", 8), (7, 1001, "f32", 3), (64, 18944, "bf16", 0),
       (300, 256, "bf16", 0)]


def glu_bounds(g, u, da):
    s = L.sigmoid(g)
    silu = np.abs(g) * s
    return 16 * U * silu * np.abs(u), 16 * U * np.abs(da * u) * (s + silu), 16 * U * np.abs(da) * silu


@pytest.mark.parametrize("rows,cols,dtype,pad", GLU)
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_swiglu(mu, rows, cols, dtype, pad, fmt):
    import torch
    wide = rand((rows, 2 * cols), dtype, 1, 4.0, pad)
    gate, up = wide[:, :cols], wide[:, cols:]
    wide[0, 0] = -200.0
    a = torch.empty((rows, cols), dtype=dt(dtype), device="cuda")
    g8, u8, a8 = (mu.Act8.empty(rows, cols, fmt) for _ in range(3))
    mu.swiglu_forward(gate, up, a, saved_gate=g8, saved_up=u8, saved_out=a8)
    g, u = f64(gate), f64(up)
    want = L.swiglu(g, u)
    close(a, want, glu_bounds(g, u, u)[0] + 1e-30)
    for x, q in ((g, g8), (u, u8)):
        assert np.array_equal(held(q)[0], L.pack(x, fmt)[0]) and np.array_equal(held(q)[1], L.pack(x, fmt)[1])
    if dtype == "f32":
        assert np.array_equal(held(a8)[0], L.pack(f64(a), fmt)[0]) and np.array_equal(held(a8)[1], L.pack(f64(a), fmt)[1])

    da = rand((rows, cols), dtype, 2, 0.1, pad)
    dgu = torch.empty((rows, 2 * cols), dtype=dt(dtype), device="cuda")
    b8 = mu.Act8.empty(rows, cols, fmt)
    mu.swiglu_backward(da, g8, u8, dgu[:, :cols], dgu[:, cols:], saved_out=b8)
    g, u, d = values(g8), values(u8), f64(da)
    dg, du = L.swiglu_grad(d, g, u)
    _, bg, bu = glu_bounds(g, u, d)
    close(dgu[:, :cols], dg, bg + 1e-30)
    close(dgu[:, cols:], du, bu + 1e-30)
    v64 = L.swiglu(g, u)
    s = np.repeat(np.exp2(L.pack(v64, fmt)[1].astype(np.float64) - 127), 32, 1)[:, :cols]
    half = 0.5 * s if fmt == "int8" else np.maximum(np.abs(v64) / 16, 2.0 ** -10 * s)
    assert np.max(np.abs(values(b8) - v64) - half * 1.001 - 32 * U * np.abs(v64) - 1e-30) <= 0
    # in place, and without the optional output
    da1, dup = da.contiguous().clone(), torch.empty((rows, cols), dtype=dt(dtype), device="cuda")
    mu.swiglu_backward(da1, g8, u8, da1, dup)
    assert torch.equal(da1, dgu[:, :cols]) and torch.equal(dup, dgu[:, cols:])


# ------------------------------------------------------------------ weight gradient
WG = [(1, 1, 1), (3, 5, 7), (63, 128, 32), (64, 128, 128), (65, 130, 129), (257, 515, 1001), (128, 256, 256),
      (1000, 512, 3584), (300, 264, 40), (2048, 257, 136), (129, 8, 2000)]


def wgrad_check(mu, plan, tokens, m, n, fmt, dtype, accumulate, scaled, pad=0):
    import torch
    dy = rand((tokens, m), "bf16", 1, 0.5, pad)
    x8 = filled(mu, rand((tokens, n), "f32", 2, 2.0), fmt)
    s = 1 + 0.3 * rand((1, n), "f32", 3)[0] if scaled else None
    g = rand((m, n), dtype, 4).contiguous()
    g0 = f64(g) if accumulate else 0.0
    plan.wgrad(dy, x8, g, col_scale=s, accumulate=accumulate)
    plan.sync()
    s64 = f64(s) if scaled else 1.0
    d, x = f64(dy), values(x8)
    want = d.T @ x * s64 + g0
    bound = 2 * (tokens + 8) * U * (np.abs(d).T @ np.abs(x)) * np.abs(s64) + 4 * U * (np.abs(want) + np.abs(g0))
    close(g, want, bound + 1e-30)


@pytest.mark.parametrize("tokens,m,n", WG)
@pytest.mark.parametrize("fmt,dtype,accumulate,scaled", [("e4m3", "bf16", False, True), ("int8", "f32", True, False),
                                                         ("e4m3", "f32", False, False), ("int8", "bf16", True, True)])
def test_wgrad(mu, plan, tokens, m, n, fmt, dtype, accumulate, scaled):
    wgrad_check(mu, plan, tokens, m, n, fmt, dtype, accumulate, scaled)


@pytest.mark.parametrize("m,n", [(300, 392), (257, 391), (64, 96)])
@pytest.mark.parametrize("dtype,accumulate", [("f32", False), ("f32", True), ("bf16", False), ("bf16", True)])
def test_wgrad_long(mu, plan, m, n, dtype, accumulate):
    """Few tiles and many tokens: tiles split along the tokens and joined, fp32 sums in several chains."""
    wgrad_check(mu, plan, 8203, m, n, "e4m3", dtype, accumulate, True)


def test_wgrad_many_experts(mu, plan):
    """More experts than are dealt out by length, and more tiles per CTA pair than are decoded at the start."""
    import torch
    e, m, n, tokens = 301, 1288, 1296, 3010            # 36 tiles each: 10836 tiles, over 96 turns of 76 pairs
    edges = [10 * i for i in range(e)] + [tokens]
    edges[5] = edges[4]                                # one without tokens, its neighbour with twenty
    dy, x8 = rand((tokens, m), "bf16", 1, 0.5), filled(mu, rand((tokens, n), "f32", 2), "int8")
    g = torch.empty((e, m, n), dtype=torch.bfloat16, device="cuda")
    plan.wgrad(dy, x8, g, offsets=torch.tensor(edges, dtype=torch.int32, device="cuda"))
    plan.sync()
    d, v = f64(dy), values(x8)
    for k in (0, 4, 5, 150, 299, 300):
        a, b = edges[k], edges[k + 1]
        close(g[k], d[a:b].T @ v[a:b], 60 * U * (np.abs(d[a:b]).T @ np.abs(v[a:b])) + 1e-30)
    whole = torch.zeros((m, n), dtype=torch.float64, device="cuda")
    for part in g.split(16):
        whole += part.double().sum(0)
    want = torch.from_numpy(d.T @ v).cuda()
    assert float((whole - want).norm() / want.norm()) < 2.0 ** -8   # bf16 roundings of the parts


@pytest.mark.parametrize("pad", [1, 4, 8])
def test_wgrad_strided_dy(mu, plan, pad):
    wgrad_check(mu, plan, 200, 320, 288, "int8", "f32", False, True, pad)


@pytest.mark.parametrize("edges,m,n", [([0, 0, 5, 5, 70, 200, 200], 136, 96), ([10, 40, 41, 150], 257, 136),
                                       ([0, 64, 128, 200], 256, 512), ([0, 200], 33, 65), ([200, 200], 16, 16)])
@pytest.mark.parametrize("dtype,accumulate", [("f32", False), ("bf16", True)])
def test_wgrad_experts(mu, plan, edges, m, n, dtype, accumulate):
    """Ragged and empty experts; the tokens outside every expert hold NaN in dy and in x."""
    import torch
    tokens, e = 200, len(edges) - 1
    dy, x = rand((tokens, m), "bf16", 1, 0.5), rand((tokens, n), "f32", 2)
    x8 = filled(mu, x, "e4m3")
    d, xv = f64(dy), values(x8)
    out = torch.ones(tokens, dtype=torch.bool)
    for a, b in zip(edges, edges[1:]):
        out[a:b] = False
    dy[out.cuda()] = float("nan")
    x8.scales[out.cuda()] = 255
    off = torch.tensor(edges, dtype=torch.int32, device="cuda")
    g = rand((e * m, n), dtype, 4).contiguous().view(e, m, n)
    g0 = f64(g) if accumulate else 0.0
    plan.wgrad(dy, x8, g, offsets=off, accumulate=accumulate)
    plan.sync()
    want = L.wgrad(d, xv, None, edges) + g0
    bound = 2 * (tokens + 8) * U * L.wgrad(np.abs(d), np.abs(xv), None, edges) + 4 * U * (np.abs(want) + np.abs(g0))
    close(g, want, bound + 1e-30)


def test_wgrad_neighbours_do_not_leak(mu, plan):
    """Each expert's gradient stays finite although the next expert's tokens hold NaN."""
    import torch
    dy, x = rand((96, 256), "bf16", 1), rand((96, 256), "f32", 2)
    dy[40:] = float("nan")
    off = torch.tensor([0, 40, 96], dtype=torch.int32, device="cuda")
    g = torch.empty((2, 256, 256), device="cuda")
    plan.wgrad(dy, filled(mu, x, "int8"), g, offsets=off)
    plan.sync()
    assert g[0].isfinite().all() and g[1].isnan().all()


def test_wgrad_bad_offsets_stay_in_bounds(mu, plan):
    """Offsets beyond the tokens are clamped, decreasing ones leave an empty expert."""
    import torch
    dy, x8 = rand((50, 64), "bf16", 1), filled(mu, rand((50, 96), "f32", 2), "int8")
    g = torch.empty((3, 64, 96), device="cuda")
    plan.wgrad(dy, x8, g, offsets=torch.tensor([-5, 20, 10, 1000], dtype=torch.int32, device="cuda"))
    plan.sync()
    want = L.wgrad(f64(dy), values(x8), None, [0, 20, 20, 50])
    want[2] = L.wgrad(f64(dy)[10:], values(x8)[10:])
    close(g, want, 200 * U * (np.abs(f64(dy)).T @ np.abs(values(x8))))


def test_same_inputs_give_the_same_bits(mu, plan):
    import torch
    dy, x8 = rand((3000, 384), "bf16", 1), filled(mu, rand((3000, 640), "f32", 2), "e4m3")
    w, rstd = torch.ones(640, device="cuda"), torch.ones(3000, device="cuda")
    d2 = rand((3000, 640), "bf16", 3)
    seen = []
    for _ in range(3):
        g, dx, dw = torch.empty((384, 640), device="cuda"), torch.empty_like(d2), torch.empty(640, device="cuda")
        plan.wgrad(dy, x8, g)
        plan.rmsnorm_backward(d2, w, rstd, dx, dw, saved=x8)
        seen.append((g, dx, dw))
    plan.sync()
    for s in seen[1:]:
        assert all(torch.equal(a, b) for a, b in zip(s, seen[0]))


def test_side_stream(mu, plan):
    """Work on a stream of the caller's, ordered by it alone."""
    import torch
    s = torch.cuda.Stream()
    x, dy = rand((512, 1024), "bf16", 1, 2.0), rand((512, 256), "bf16", 2)
    w = torch.ones(1024, device="cuda")
    ref, out = torch.empty((256, 1024), device="cuda"), torch.empty((256, 1024), device="cuda")
    for stream, g in ((None, ref), (s, out)):
        torch.cuda.synchronize()
        a = mu.Act8.empty(512, 1024)
        mu.rmsnorm_forward(x, w, 1e-6, saved=a, stream=stream)
        plan.wgrad(dy, a, g, col_scale=w, stream=stream)
        plan.sync(stream)
    assert torch.equal(ref, out)


def test_long_pitch_offsets_pass_32_bits(mu, plan):
    """Rows whose byte offsets pass 2^32: a column block of a tensor with a pitch of 2^21 elements."""
    import torch
    wide = torch.empty((1100, 1 << 21), dtype=torch.bfloat16, device="cuda")   # 4.6 GB
    x = wide[:, 64:64 + 320].copy_(rand((1100, 320), "bf16", 1))
    a, y = filled(mu, x, "int8"), wide[:, 1024:1024 + 320]
    mu.act_unpack(a, y)
    assert np.array_equal(held(a)[0], L.pack(f64(x), "int8")[0]) and np.array_equal(f64(y), values(a))
    g = torch.empty((320, 320), device="cuda")
    plan.wgrad(x, a, g)
    plan.sync()
    d, v = f64(x), values(a)
    close(g, d.T @ v, 2 * 1108 * U * (np.abs(d).T @ np.abs(v)))

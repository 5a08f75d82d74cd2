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

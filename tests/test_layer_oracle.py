"""Pins of the layer-side fp64 definitions (oracle/layer_ref.py), on the CPU: the 8-bit
format against exhaustive search, the gradients against differences."""
import numpy as np
import pytest

from oracle import layer_ref as L


def test_e4m3_numbers_of_the_format():
    assert L.e4m3_number(0x7E) == 448 and L.e4m3_number(0x01) == 2.0 ** -9 and L.e4m3_number(0x38) == 1
    assert np.isnan(L.e4m3_number(0x7F)) and L.e4m3_number(0xB8) == -1
    assert np.all(np.diff(L._E4M3) > 0)


def test_e4m3_code_is_the_nearest_with_ties_to_even():
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.standard_normal(2000) * 30, (L._E4M3[:-1] + L._E4M3[1:]) / 2, L._E4M3, [448, 1e9, -1e9]])
    q = L.e4m3_code(x)
    v = L.e4m3_number(q)
    best = np.min(np.abs(np.abs(x)[:, None] - L._E4M3[None]), 1)
    assert np.array_equal(np.abs(np.abs(x) - np.abs(v)), best)
    mid = L.e4m3_code((L._E4M3[:-1] + L._E4M3[1:]) / 2)
    assert np.all(mid % 2 == 0)


def test_torch_agrees_on_e4m3_codes():
    torch = pytest.importorskip("torch")
    x = np.random.default_rng(1).standard_normal(5000).astype(np.float32) * 100
    x = np.clip(x, -448, 448)
    assert np.array_equal(L.e4m3_code(x.astype(np.float64)),
                          torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_scale_is_the_smallest_that_fits(fmt):
    top = L.LARGEST[fmt]
    for amax in [1.0, top, top * (1 + 2.0 ** -23), top * (1 - 2.0 ** -23), 1e-20, 3.0, 2.0 ** 60, top * 2.0 ** 100]:
        e = int(L.scale_exponent(np.array([amax]), fmt)[0])
        assert amax <= top * 2.0 ** e and amax > top * 2.0 ** (e - 1)
    assert L.scale_exponent(np.array([0.0]), fmt)[0] == L.LOWEST_EXP
    assert L.scale_exponent(np.array([3.38e38]), fmt)[0] == L.HIGHEST_EXP[fmt]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_pack_marks_groups_that_are_not_finite(fmt):
    x = np.ones((2, 70))
    x[0, 33], x[1, 69] = np.inf, np.nan
    q, s = L.pack(x, fmt)
    v = L.unpack(q, s, fmt)
    assert np.isnan(v[0, 32:64]).all() and np.isfinite(v[0, :32]).all() and np.isfinite(v[0, 64:]).all()
    assert np.isnan(v[1, 64:]).all() and np.array_equal(v[1, :64], x[1, :64])


def test_every_value_is_a_bf16_number():
    torch = pytest.importorskip("torch")
    x = np.random.default_rng(2).standard_normal((64, 320)) * np.exp2(np.linspace(-120, 120, 64))[:, None]
    for fmt in ("e4m3", "int8"):
        v = L.unpack(*L.pack(x.astype(np.float32), fmt), fmt)
        assert np.array_equal(torch.from_numpy(v).to(torch.bfloat16).double().numpy(), v)


def _difference(f, x, d, step=1e-5):
    return (f(x + step * d) - f(x - step * d)) / (2 * step)


def test_rmsnorm_gradient_against_differences():
    rng = np.random.default_rng(3)
    x, r, w, dy, dres = (rng.standard_normal(s) for s in [(5, 37), (5, 37), (37,), (5, 37), (5, 37)])
    h, _, xhat, rstd = L.rmsnorm(x, w, 1e-6, r)
    dh, dw = L.rmsnorm_grad(dy, xhat, rstd, w, dres)
    for _ in range(5):
        d = rng.standard_normal((5, 37))
        slope = _difference(lambda z: np.sum(L.rmsnorm(z, w, 1e-6, r)[1] * dy) + np.sum((z + r) * dres), x, d)
        assert abs(slope - np.sum(dh * d)) < 1e-7 * (1 + abs(slope))
        e = rng.standard_normal(37)
        slope = _difference(lambda z: np.sum(L.rmsnorm(x, z, 1e-6, r)[1] * dy), w, e)
        assert abs(slope - np.sum(dw * e)) < 1e-7 * (1 + abs(slope))


def test_swiglu_gradient_against_differences():
    rng = np.random.default_rng(4)
    g, u, da = (rng.standard_normal((6, 21)) * 3 for _ in range(3))
    dg, du = L.swiglu_grad(da, g, u)
    for _ in range(5):
        d = rng.standard_normal((6, 21))
        for f, x, grad in ((lambda z: np.sum(L.swiglu(z, u) * da), g, dg), (lambda z: np.sum(L.swiglu(g, z) * da), u, du)):
            slope = _difference(f, x, d)
            assert abs(slope - np.sum(grad * d)) < 1e-7 * (1 + abs(slope))


def test_wgrad_is_the_gradient_of_the_product():
    rng = np.random.default_rng(5)
    x, w, dy, s = (rng.standard_normal(k) for k in [(9, 7), (4, 7), (9, 4), (7,)])
    g = L.wgrad(dy, x, s)
    d = rng.standard_normal((4, 7))
    slope = _difference(lambda z: np.sum(((x * s) @ z.T) * dy), w, d)
    assert abs(slope - np.sum(g * d)) < 1e-7 * (1 + abs(slope))
    parts = L.wgrad(dy, x, None, [0, 3, 3, 9])
    assert np.allclose(parts.sum(0), dy.T @ x) and not parts[1].any()

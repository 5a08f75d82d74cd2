"""The norm of all gradients and their clipping on the GPU against fp64.

The squares of up to 64 values are summed in fp32 (19 roundings of 2^-24 on any way at most), the rest in fp64; the norm
is the root, so half of that, and one rounding to fp32: below 18 u.  Scaling: the factor is one fp32 division of the rounded norm,
the product one rounding, then the output type's own: within 2.5 u (fp32) of g max_norm / norm as the call read the norm."""
import numpy as np
import pytest

from test_gpu_layer import U, close, dt, f64, mu, plan  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu
TOL = 18 * U


def tensors(sizes, dtypes, seed=0, scale=1e-3, shift=0):
    """Tensors in one buffer each, `shift` elements into it."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for n, d in zip(sizes, dtypes):
        buf = (torch.randn(n + shift, generator=g, device="cuda") * scale).to(dt(d))
        out.append(buf[shift:])
    return out


def norm64(ts):
    return float(np.sqrt(sum(float((t.double() ** 2).sum()) for t in ts)))


def norm_of(plan, ts):  # noqa: F811
    import torch
    n = torch.full((1,), -1.0, device="cuda")
    plan.grad_norm(ts, n)
    return float(n)


CASES = [([1], ["f32"]), ([1], ["bf16"]), ([7, 9], ["bf16", "f32"]), ([8192], ["bf16"]), ([8193, 5], ["f32", "bf16"]),
         ([100000, 1, 0, 77777, 0], ["bf16", "f32", "bf16", "f32", "bf16"]), ([3, 4] * 20, ["bf16", "f32"] * 20),
         (list(range(1, 2700)), ["bf16", "f32", "bf16"] * 900), ([5000000], ["bf16"]), ([0, 0], ["f32", "bf16"])]


@pytest.mark.parametrize("shift", [0, 1, 3])
@pytest.mark.parametrize("sizes,dtypes", CASES)
def test_norm(plan, sizes, dtypes, shift):  # noqa: F811
    ts = tensors(sizes, dtypes, shift=shift)
    want = norm64(ts)
    assert abs(norm_of(plan, ts) - want) <= TOL * want
    assert norm_of(plan, ts) == norm_of(plan, ts)   # the same bits


def test_norm_of_nothing(plan):  # noqa: F811
    import torch
    assert norm_of(plan, []) == 0.0
    assert norm_of(plan, [torch.zeros(100000, device="cuda"), torch.zeros(5, device="cuda").bfloat16()]) == 0.0


@pytest.mark.parametrize("scale", [1e-44, 1e-38, 1e-30, 1e-22, 1e-14, 1e10, 1e19, 1e25, 1e30])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_squares_neither_overflow_nor_vanish(plan, dtype, scale):  # noqa: F811
    import torch
    g = torch.Generator(device="cuda").manual_seed(3)
    t = (torch.randn(70001, generator=g, device="cuda", dtype=torch.float64) * scale).to(dt(dtype))
    want = norm64([t])
    # a norm below the normal range is rounded to a multiple of 2^-149
    assert abs(norm_of(plan, [t]) - want) <= TOL * want + 2.0 ** -150


def test_large_and_tiny_values_together(plan):  # noqa: F811
    import torch
    t = torch.full((40000,), 1e-25, device="cuda")
    t[::7] = 1e-10
    t[12345] = 3e20
    u = torch.full((40000,), 1e-25, device="cuda")
    assert abs(norm_of(plan, [t, u]) - norm64([t, u])) <= TOL * norm64([t, u])
    assert abs(norm_of(plan, [u]) - norm64([u])) <= TOL * norm64([u])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_norm_of_what_is_not_finite(plan, dtype):  # noqa: F811
    import torch
    t = tensors([50000], [dtype])[0]
    t[777] = float("inf")
    assert norm_of(plan, [t]) == float("inf")
    t[49999] = float("nan")
    assert np.isnan(norm_of(plan, [t]))
    big = torch.full((1000,), 3e38, device="cuda").to(dt(dtype))   # a norm beyond fp32
    assert norm_of(plan, [big]) == float("inf")


def test_norm_of_many_values_of_one_size(plan):  # noqa: F811
    """2^28 equal values: long sums do not drift."""
    import torch
    t = torch.full((1 << 28,), 0.37, device="cuda").bfloat16()
    want = float(t[0].double()) * 2 ** 14
    assert abs(norm_of(plan, [t]) - want) <= TOL * want


@pytest.mark.parametrize("max_norm", [0.01, 1e6])
@pytest.mark.parametrize("shift", [0, 1, 2, 5])
@pytest.mark.parametrize("out", ["in place", "same", "f32", "bf16"])
def test_clip(plan, out, shift, max_norm):  # noqa: F811
    import torch
    sizes, dtypes = [1, 8, 65536, 70001, 0, 33, 9], ["f32", "bf16", "bf16", "f32", "f32", "bf16", "bf16"]
    ts = tensors(sizes, dtypes, seed=4, shift=shift)
    keep = [t.clone() for t in ts]
    edges = [t._base[:shift].clone() if shift else None for t in ts]
    norm = torch.zeros(1, device="cuda")
    plan.grad_norm(ts, norm)
    n = float(norm)
    if out == "in place":
        plan.grad_clip(ts, norm, max_norm)
        got = ts
    else:
        kinds = dtypes if out == "same" else [out] * len(ts)
        got = [torch.full((s + 9 - shift,), 5.0, dtype=dt(k), device="cuda")[9 - shift:] for s, k in zip(sizes, kinds)]
        plan.grad_clip(ts, norm, max_norm, out=got)
        for g, s in zip(got, sizes):
            assert bool((g._base[:9 - shift] == 5).all()) if g._base is not None else True
        assert all(torch.equal(a, b) for a, b in zip(ts, keep))
    f = max_norm / n if n > max_norm else 1.0
    for g, k, s in zip(got, keep, sizes):
        if s == 0:
            continue
        if f == 1.0 and g.dtype == k.dtype:
            assert torch.equal(g, k)
        close(g, f64(k) * f, 2.5 * U * np.abs(f64(k) * f) * (f != 1.0) + 2.0 ** -149)
    if shift and out == "in place":
        assert all(torch.equal(t._base[:shift], e) for t, e in zip(ts, edges))


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_a_norm_that_is_not_finite_leaves_the_gradients(plan, bad):  # noqa: F811
    import torch
    ts = tensors([5000, 300], ["bf16", "f32"])
    ts[0][17] = bad
    keep = [t.clone() for t in ts]
    norm = torch.zeros(1, device="cuda")
    plan.grad_norm(ts, norm)
    plan.grad_clip(ts, norm, 1e-4)
    for t, k in zip(ts, keep):
        assert torch.equal(t.nan_to_num(nan=7.0), k.nan_to_num(nan=7.0))


def test_clip_into_the_type_of_the_step(mu, plan):  # noqa: F811
    """fp32 sums clipped into bf16 gradients, then a step: as with gradients clipped by hand."""
    import torch
    shapes = [(200, 300), (136, 512)]
    g = torch.Generator(device="cuda").manual_seed(1)
    sums = [torch.randn(s, generator=g, device="cuda") for s in shapes]
    low = [torch.empty(s, dtype=torch.bfloat16, device="cuda") for s in shapes]
    norm = torch.zeros(1, device="cuda")
    plan.grad_norm(sums, norm)
    plan.grad_clip(sums, norm, 1.0, out=low)
    by_hand = [(s * (1.0 / norm)).bfloat16() for s in sums]
    # the factor is the same fp32 division here: 1 / norm
    assert all(torch.equal(a, b) for a, b in zip(low, by_hand))
    W = [[torch.ones(s, device="cuda") * 0.1 for s in shapes] for _ in range(2)]
    M = [[torch.zeros(s, device="cuda") for s in shapes] for _ in range(2)]
    with mu.MuonPlan(shapes, "bf16") as p:
        p.step(W[0], low, M[0], 0.02, 0.1)
        p.step(W[1], by_hand, M[1], 0.02, 0.1)
        p.sync()
    assert all(torch.equal(a, b) for a, b in zip(W[0] + M[0], W[1] + M[1]))


def test_captured(mu, plan):  # noqa: F811
    import torch
    ts = tensors([100000, 3333] + [50] * 1200, ["bf16", "f32"] + ["bf16"] * 1200)
    grads, norm = mu.GradList(ts), torch.zeros(1, device="cuda")
    plan.grad_norm(grads, norm)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.grad_norm(grads, norm)
        plan.grad_clip(grads, norm, 0.5)
    for scale in (1.0, 1e-6, 30.0):
        new = tensors([100000, 3333] + [50] * 1200, ["bf16", "f32"] + ["bf16"] * 1200, seed=9, scale=scale)
        for t, x in zip(ts, new):
            t.copy_(x)
        graph.replay()
        want = norm64(new)
        assert abs(float(norm) - want) <= TOL * want
        # bf16 results: each rounded to 2^-9 of itself
        assert abs(norm64(ts) - min(want, 0.5)) <= 2.0 ** -8 * min(want, 0.5)


def test_what_the_binding_refuses(mu, plan):  # noqa: F811
    import torch
    a, b = torch.zeros(10, device="cuda"), torch.zeros(20, device="cuda").bfloat16()
    norm = torch.zeros(1, device="cuda")
    for call in (lambda: mu.GradList([a.half()]), lambda: mu.GradList([a.cpu()]), lambda: mu.GradList([b.view(4, 5).t()]),
                 lambda: plan.grad_norm([a], torch.zeros(2, device="cuda")), lambda: plan.grad_norm([a], norm.double()),
                 lambda: plan.grad_clip([a, b], norm, 1.0, out=[b, a]), lambda: plan.grad_clip([a, b], norm, 1.0, out=[a])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: plan.grad_clip([a, a], norm, 1.0), lambda: plan.grad_clip([a, a[5:]], norm, 1.0),
                 lambda: plan.grad_clip([a], norm, 0.0), lambda: plan.grad_clip([a, norm], norm, 1.0),
                 lambda: plan.grad_clip([a], norm, 1.0, out=[a.view(torch.bfloat16)[:10]])):
        with pytest.raises(mu.MuonError):
            call()

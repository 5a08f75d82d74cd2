"""The order of tokens by expert and the moves of their rows on the GPU.

The order and the copies are exact.  With u = 2^-24: the weighted sum of k rows carries (k + 1) u of its terms'
magnitudes, a dot product of C terms (C + 8) u; a bf16 output lies between the bf16 roundings of the interval's ends."""
import numpy as np
import pytest

from test_gpu_layer import U, close, dt, f64, mu, rand  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu


def order(ids, experts):
    """The definition: (offsets, slots)."""
    flat = ids.reshape(-1)
    slots, offsets, place = np.full(flat.shape, -1), np.zeros(experts + 1, int), 0
    for e in range(experts):
        at = np.nonzero(flat == e)[0]
        slots[at] = place + np.arange(at.size)
        place += at.size
        offsets[e + 1] = place
    return offsets, slots.reshape(ids.shape)


def ordered(mu, ids, experts, **kw):  # noqa: F811
    import torch
    t = torch.tensor(ids, dtype=torch.int32, device="cuda")
    offsets = torch.full((experts + 1,), -7, dtype=torch.int32, device="cuda")
    slots = torch.full_like(t, -7)
    mu.expert_order(t, offsets, slots, **kw)
    return offsets, slots


@pytest.mark.parametrize("tokens,choices,experts", [(1, 1, 1), (1, 8, 32), (0, 4, 16), (7, 3, 5), (33, 2, 2), (1000, 8, 128),
                                                    (1025, 7, 64), (4097, 2, 300), (1200, 64, 4096), (9001, 3, 1025),
                                                    (30000, 8, 256), (100003, 1, 3), (5000, 2, 2049)])
@pytest.mark.parametrize("kind", ["even", "skewed", "one", "none"])
def test_order(mu, tokens, choices, experts, kind):  # noqa: F811
    rng = np.random.default_rng(tokens + experts)
    ids = rng.integers(0, experts, (tokens, choices))
    if kind == "skewed":
        ids = np.minimum((rng.random((tokens, choices)) ** 6 * experts).astype(int), experts - 1)
        ids[rng.random((tokens, choices)) < 0.2] = -1
        ids[rng.random((tokens, choices)) < 0.05] = experts + rng.integers(0, 1000)
    elif kind == "one":
        ids[:] = experts - 1
    elif kind == "none":
        ids[:] = -1
    offsets, slots = ordered(mu, ids, experts)
    want = order(ids, experts)
    assert np.array_equal(offsets.cpu().numpy(), want[0])
    assert np.array_equal(slots.cpu().numpy(), want[1])


def test_order_of_extreme_ids(mu):  # noqa: F811
    ids = np.array([[2 ** 31 - 1, -2 ** 31, 3, 0], [4, 3, 2, -1]])
    offsets, slots = ordered(mu, ids, 4)
    want = order(ids, 4)
    assert np.array_equal(offsets.cpu().numpy(), want[0]) and np.array_equal(slots.cpu().numpy(), want[1])


SHAPES = [(1, 1, 1, 0), (1, 8, 64, 0), (5, 3, 31, 1), (40, 4, 256, 8), (65, 2, 1001, 3), (130, 8, 264, 0), (9, 5, 5000, 0),
          (2, 64, 40, 0), (333, 3, 513, 5), (17, 2, 8192, 0)]


def routed(tokens, choices, seed, experts=16):
    """Slots with padding tokens, and the number of rows with a few behind the last."""
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, experts, (tokens, choices))
    ids[rng.random((tokens, choices)) < 0.15] = -1
    return order(ids, experts)[1], tokens * choices + 3


def on_gpu(a, dtype=None):
    import torch
    return torch.tensor(a, dtype=dtype or torch.int32, device="cuda")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens,choices,cols,pad", SHAPES)
def test_dispatch(mu, dtype, tokens, choices, cols, pad):  # noqa: F811
    import torch
    slots, rows = routed(tokens, choices, tokens + cols)
    x = rand((tokens, cols), dtype, 1, pad=pad)
    wide = torch.full((rows, cols + 2 * pad), 9.0, dtype=dt(dtype), device="cuda")
    mu.expert_dispatch(x, on_gpu(slots), wide[:, pad:pad + cols])
    want = np.full((rows, cols + 2 * pad), 9.0)
    for t, j in zip(*np.nonzero(slots >= 0)):
        want[slots[t, j], pad:pad + cols] = f64(x)[t]
    assert np.array_equal(f64(wide), want)


def test_dispatch_copies_bits(mu):  # noqa: F811
    """NaNs of any payload, infinities, zeros of either sign and subnormal numbers arrive as they were."""
    import torch
    bits = torch.arange(-32768, 32768, device="cuda").to(torch.int16).view(64, 1024)
    slots = on_gpu(np.random.default_rng(0).permutation(64).reshape(64, 1))
    for lead in (0, 1):
        x = torch.zeros((64, 1025), dtype=torch.int16, device="cuda")[:, lead:lead + 1024]
        x.copy_(bits)
        out = torch.zeros((64, 1025), dtype=torch.bfloat16, device="cuda")[:, lead:lead + 1024]
        mu.expert_dispatch(x.view(torch.bfloat16), slots, out)
        assert torch.equal(out.view(torch.int16)[slots[:, 0].long()], bits)


@pytest.mark.parametrize("weighted", [True, False])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens,choices,cols,pad", SHAPES)
def test_combine(mu, dtype, tokens, choices, cols, pad, weighted):  # noqa: F811
    import torch
    slots, rows = routed(tokens, choices, tokens + cols)
    r = rand((rows, cols), dtype, 2, pad=pad)
    r[rows - 3:] = float("nan")          # rows that no token stands in
    w = torch.rand((tokens, choices), device="cuda") if weighted else None
    wide = torch.full((tokens, cols + 2 * pad), 9.0, dtype=dt(dtype), device="cuda")
    mu.expert_combine(r, on_gpu(slots), wide[:, pad:pad + cols], weights=w)
    there = (slots >= 0)[:, :, None]
    terms = np.where(there, f64(r)[np.maximum(slots, 0)] * (f64(w)[:, :, None] if weighted else 1.0), 0.0)
    close(wide[:, pad:pad + cols], terms.sum(1), (choices + 1) * U * np.abs(terms).sum(1))
    edges = torch.cat([wide[:, :pad], wide[:, pad + cols:]], 1)
    assert bool((edges == 9).all())


@pytest.mark.parametrize("outputs", ["both", "drows", "dweights"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("tokens,choices,cols,pad", SHAPES)
def test_combine_backward(mu, dtype, tokens, choices, cols, pad, outputs):  # noqa: F811
    import torch
    slots, rows = routed(tokens, choices, tokens + cols)
    r = rand((rows, cols), dtype, 3, pad=pad)
    r[rows - 3:] = float("nan")
    d = rand((tokens, cols), dtype, 4, pad=pad)
    w = torch.rand((tokens, choices), device="cuda")
    wide = torch.full((rows, cols + 2 * pad), 9.0, dtype=dt(dtype), device="cuda")
    drows = wide[:, pad:pad + cols] if outputs != "dweights" else None
    dw = torch.full((tokens, choices), 9.0, device="cuda") if outputs != "drows" else None
    mu.expert_combine_backward(d, on_gpu(slots), w, rows=r if outputs != "drows" else None, drows=drows, dweights=dw)
    if dw is not None:
        there = slots >= 0
        terms = np.where(there[:, :, None], f64(d)[:, None, :] * f64(r)[np.maximum(slots, 0)], 0.0)
        close(dw, terms.sum(2), (cols + 8) * U * np.abs(terms).sum(2))
    if drows is not None:
        want = np.full((rows, cols + 2 * pad), 9.0)
        bound = np.zeros_like(want)
        for t, j in zip(*np.nonzero(slots >= 0)):
            want[slots[t, j], pad:pad + cols] = f64(w)[t, j] * f64(d)[t]
            bound[slots[t, j], pad:pad + cols] = U * np.abs(f64(w)[t, j] * f64(d)[t])
        close(wide, want, bound)


def test_slots_outside_the_rows_are_no_choices(mu):  # noqa: F811
    import torch
    slots = on_gpu([[0, 5], [-1, 2 ** 31 - 1], [-2 ** 31, 1]])
    x = rand((3, 40), "f32", 5)
    out = torch.full((2, 40), 3.0, device="cuda")
    mu.expert_dispatch(x, slots, out)
    assert torch.equal(out[0], x[0]) and torch.equal(out[1], x[2])
    back = torch.full((3, 40), 3.0, device="cuda")
    mu.expert_combine(out, slots, back)
    assert torch.equal(back[0], x[0]) and bool((back[1] == 0).all()) and torch.equal(back[2], x[2])
    dw = torch.full((3, 2), 3.0, device="cuda")
    mu.expert_combine_backward(x, slots, torch.ones((3, 2), device="cuda"), rows=out, dweights=dw)
    assert [float(v) for v in dw.flatten()][1:5] == [0, 0, 0, 0]


def test_no_rows(mu):  # noqa: F811
    import torch
    none = torch.empty((0, 40), device="cuda")
    slots = on_gpu(np.zeros((3, 2)))
    mu.expert_dispatch(rand((3, 40), "f32", 5), slots, none)
    out = torch.full((3, 40), 3.0, device="cuda")
    mu.expert_combine(none, slots, out)
    assert bool((out == 0).all())
    mu.expert_dispatch(none, torch.empty((0, 2), dtype=torch.int32, device="cuda"), rand((3, 40), "f32", 5))
    mu.expert_combine(rand((3, 40), "f32", 5), torch.empty((0, 2), dtype=torch.int32, device="cuda"), none)


def test_moves_are_each_others_gradients(mu):  # noqa: F811
    """<combine(dispatch(x)), g> against the backward calls, by differences in fp64: both are linear."""
    import torch
    tokens, choices, cols = 50, 4, 333
    slots, rows = routed(tokens, choices, 8)
    s = on_gpu(slots)
    x, g = rand((tokens, cols), "f32", 6), rand((tokens, cols), "f32", 7)
    w = torch.rand((tokens, choices), device="cuda")
    xs, y = torch.zeros((rows, cols), device="cuda"), torch.empty((tokens, cols), device="cuda")
    mu.expert_dispatch(x, s, xs)
    mu.expert_combine(xs, s, y, weights=w)
    drows, dw, dx = torch.zeros_like(xs), torch.empty_like(w), torch.empty_like(x)
    mu.expert_combine_backward(g, s, w, rows=xs, drows=drows, dweights=dw)
    mu.expert_combine(drows, s, dx)
    there = torch.tensor(slots >= 0, device="cuda").double()

    def loss(x_, w_):
        return float(((w_ * there).sum(1, keepdim=True) * x_ * g.double()).sum())
    vx, vw = rand((tokens, cols), "f32", 8).double(), torch.rand((tokens, choices), device="cuda").double()
    x64, w64 = x.double(), w.double()
    size = float((x64.abs() * g.double().abs()).sum()) * 2 * choices + float((vx.abs() * g.double().abs()).sum()) * choices
    assert abs(loss(x64 + vx, w64) - loss(x64, w64) - float((dx.double() * vx).sum())) <= (cols + 16) * U * size
    assert abs(loss(x64, w64 + vw) - loss(x64, w64) - float((dw.double() * vw).sum())) <= (cols + 16) * U * size


def test_captured(mu):  # noqa: F811
    import torch
    rng = np.random.default_rng(1)
    ids = on_gpu(rng.integers(0, 32, (3000, 4)))
    offsets, slots = torch.empty(33, dtype=torch.int32, device="cuda"), torch.empty_like(ids)
    x, xs, y = rand((3000, 200), "bf16", 1), torch.zeros((12000, 200), dtype=torch.bfloat16, device="cuda"), \
        torch.empty((3000, 200), dtype=torch.bfloat16, device="cuda")

    def step():
        mu.expert_order(ids, offsets, slots)
        mu.expert_dispatch(x, slots, xs)
        mu.expert_combine(xs, slots, y)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3):
        new = rng.integers(-1, 33, (3000, 4))
        ids.copy_(on_gpu(new))
        graph.replay()
        want = order(new, 32)
        assert np.array_equal(offsets.cpu().numpy(), want[0]) and np.array_equal(slots.cpu().numpy(), want[1])
        count = torch.tensor((want[1] >= 0).sum(1), device="cuda")[:, None]
        # up to four copies: exact in fp32 (8 + 2 bits), rounded once
        assert torch.equal(y, (x.float() * count).bfloat16())


def test_on_another_stream(mu):  # noqa: F811
    """The calls run on the stream that they are given, behind what is on it."""
    import torch
    ids = on_gpu(np.random.default_rng(2).integers(0, 16, (2000, 3)))
    x = rand((2000, 300), "bf16", 1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        big = torch.randn(4096, 4096, device="cuda")
        for _ in range(3):
            big = big @ big / 64           # what comes before on that stream
        new = x * 2
    offsets, slots = torch.empty(17, dtype=torch.int32, device="cuda"), torch.empty_like(ids)
    xs, y, dw = torch.zeros((6000, 300), dtype=torch.bfloat16, device="cuda"), torch.empty_like(x), \
        torch.empty((2000, 3), device="cuda")
    ones = torch.ones((2000, 3), device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    mu.expert_order(ids, offsets, slots, stream=s)
    mu.expert_dispatch(new, slots, xs, stream=s)
    mu.expert_combine(xs, slots, y, stream=s)
    mu.expert_combine_backward(y, slots, ones, rows=xs, dweights=dw, stream=s)
    s.synchronize()
    assert torch.equal(y, (x.float() * 6).bfloat16())   # three copies of 2 x
    want = order(ids.cpu().numpy(), 16)
    assert np.array_equal(slots.cpu().numpy(), want[1])
    assert torch.allclose(dw, (y.float() * new.float()).sum(1, keepdim=True).expand(-1, 3), rtol=1e-4, atol=1e-3)


def test_what_the_binding_refuses(mu):  # noqa: F811
    import torch
    ids, slots = on_gpu(np.zeros((8, 2))), on_gpu(np.arange(16).reshape(8, 2))
    offsets, x, rows = torch.empty(5, dtype=torch.int32, device="cuda"), rand((8, 40), "f32", 1), rand((16, 40), "f32", 2)
    w = torch.ones((8, 2), device="cuda")
    bad = [lambda: mu.expert_order(ids.long(), offsets, slots), lambda: mu.expert_order(ids[:, :1], offsets, slots),
           lambda: mu.expert_order(ids, offsets.long(), slots), lambda: mu.expert_order(ids, offsets[:1], slots),
           lambda: mu.expert_order(ids.flatten(), offsets, slots), lambda: mu.expert_order(ids.t(), offsets, slots),
           lambda: mu.expert_dispatch(x, slots[:4], rows), lambda: mu.expert_dispatch(x, slots, rows.bfloat16()),
           lambda: mu.expert_dispatch(x, slots, rows[:, :39]), lambda: mu.expert_dispatch(x.half(), slots, rows.half()),
           lambda: mu.expert_dispatch(x, slots, rows.cpu()), lambda: mu.expert_dispatch(x.t(), slots, rows),
           lambda: mu.expert_combine(rows, slots, x, weights=w.bfloat16()),
           lambda: mu.expert_combine(rows, slots, x, weights=w[:, :1]),
           lambda: mu.expert_combine_backward(x, slots, w, rows=rows, drows=rows[:8].clone()),
           lambda: mu.expert_combine_backward(x, slots, w, rows=rows, dweights=w.double())]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    for call in (lambda: mu.expert_dispatch(rows[:8], slots, rows), lambda: mu.expert_combine(rows, slots, rows[:8]),
                 lambda: mu.expert_combine_backward(x, slots, w), lambda: mu.expert_combine_backward(x, slots, w, dweights=w),
                 lambda: mu.expert_combine_backward(x, slots, w, rows=rows, drows=rows)):
        with pytest.raises(mu.MuonError):
            call()

"""The products of a weight and of experts' weights on the GPU against fp64.

Bounds, u = 2^-24: bf16 products are exact in fp32; a sum of K of them in fp32 carries at most (2 K + 8) u of the
terms' magnitudes (the tensor cores' adds truncate: 2 u each; a few more where parts of a sum are joined).  A bf16
output has to lie between the bf16 roundings of the two ends of that interval."""
import numpy as np
import pytest

from test_gpu_layer import U, mu, plan  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu


def bf16(shape, seed, scale=1.0, pad=0, lead=0):
    """N(0, scale^2) in bf16; pad, lead: a column block of a wider tensor, `lead` values from its edge."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    wide = (torch.randn(shape[:-1] + (shape[-1] + pad,), generator=g, device="cuda") * scale).bfloat16()
    return wide[..., lead:lead + shape[-1]]


def rounded(x):
    """fp64 on the GPU to the nearest bf16, ties to even (normal range): in whole numbers, the last 45 bits away."""
    import torch
    b = x.contiguous().view(torch.int64)
    return (((b + ((1 << 44) - 1) + ((b >> 45) & 1)) >> 45) << 45).view(torch.float64)


def run(plan, x, w, out, offsets, dgrad):
    (plan.dgrad if dgrad else plan.product)(x, w, out, offsets=offsets)


def ranges(edges, tokens):
    """(expert, first, end) as the documentation clamps them."""
    for e, (a, b) in enumerate(zip(edges, edges[1:])):
        a = min(max(a, 0), tokens)
        yield e, a, min(max(b, a), tokens)


def check(plan, x, w, edges, dgrad, out=None, rows=None):
    import torch
    tokens, cols = x.shape[0], w.shape[-1 if dgrad else -2]
    if out is None:
        out = torch.full((tokens, cols), 77.0, dtype=torch.bfloat16, device="cuda")
    before = out.clone()
    offsets = None if edges is None else torch.tensor(edges, dtype=torch.int32, device="cuda")
    run(plan, x, w, out, offsets, dgrad)
    plan.sync()
    claims = torch.zeros(tokens, dtype=torch.int32, device="cuda")
    spans = list(ranges(edges, tokens)) if edges is not None else [(0, 0, tokens)]
    for _, a, b in spans:
        claims[a:b] += 1
    for e, a, b in spans:
        if a == b:
            continue
        we = (w if edges is None else w[e]).double()
        we = we if dgrad else we.t()
        xe = x[a:b].double()
        want, size = xe @ we, xe.abs() @ we.abs()
        bound = (2 * xe.shape[1] + 8) * U * size
        got = out[a:b].double()
        fine = (rounded(want - bound) <= got) & (got <= rounded(want + bound))
        fine |= claims[a:b, None] > 1    # decreasing offsets: a row of two experts is either's
        assert bool(fine.all()), (e, a, b, int((~fine).sum()), float((got - want).abs().max()))
    assert torch.equal(out[claims == 0], before[claims == 0])   # rows outside every expert
    return out


SIZES = [(1, 1, 1), (3, 5, 7), (2, 8, 16), (1, 256, 64), (64, 256, 64), (33, 300, 136), (256, 256, 128), (257, 515, 1001),
         (300, 264, 1000), (31, 1024, 2048), (1000, 512, 72), (520, 770, 650)]


@pytest.mark.parametrize("dgrad", [False, True])
@pytest.mark.parametrize("tokens,m,n", SIZES)
def test_one_weight(plan, tokens, m, n, dgrad):  # noqa: F811
    check(plan, bf16((tokens, m if dgrad else n), 1), bf16((m, n), 2, 0.1), None, dgrad)


EDGES = [[0, 5], [0, 0, 1, 1, 40, 300], [0, 64, 128, 192, 256], [3, 3, 100, 101, 250], [0] * 9 + [300],
         [0, 257, 290, 300], [0, 1, 3, 6, 10, 15, 21, 28, 36, 45, 55, 66, 78, 91, 105, 120, 136, 153, 171, 190, 210],
         [0, 33, 65, 160, 300]]


@pytest.mark.parametrize("dgrad", [False, True])
@pytest.mark.parametrize("m,n", [(256, 128), (300, 72), (129, 515), (520, 1024)])
@pytest.mark.parametrize("edges", EDGES)
def test_experts(plan, edges, m, n, dgrad):  # noqa: F811
    check(plan, bf16((300, m if dgrad else n), 3), bf16((len(edges) - 1, m, n), 4, 0.1), edges, dgrad)


@pytest.mark.parametrize("dgrad", [False, True])
@pytest.mark.parametrize("edges", [[-5, 20, 10, 400], [400, 500], [0, 300, 300, 200], [-9, -3, 5]])
def test_offsets_are_clamped(plan, edges, dgrad):  # noqa: F811
    """Beyond the tokens, and ranges that begin after their end: nothing outside [0, tokens) is touched."""
    check(plan, bf16((300, 264 if dgrad else 136), 3), bf16((len(edges) - 1, 264, 136), 4, 0.1), edges, dgrad)


@pytest.mark.parametrize("groups", [9, 4096])
def test_offsets_that_go_back_and_forth(plan, groups):  # noqa: F811
    """More tokens among the experts than there are: no fault, and nothing beside the output's rows is written."""
    import torch
    tokens, m, n = 20000, 40, 24
    offsets = torch.tensor([0 if i % 2 == 0 else tokens for i in range(groups + 1)], dtype=torch.int32, device="cuda")
    wide = torch.full((tokens + 2, m), 3.0, dtype=torch.bfloat16, device="cuda")
    plan.product(bf16((tokens, n), 1), bf16((groups, m, n), 2), wide[1:-1], offsets=offsets)
    plan.sync()
    assert bool((wide[0] == 3).all()) and bool((wide[-1] == 3).all())


@pytest.mark.parametrize("dgrad", [False, True])
@pytest.mark.parametrize("pad,lead", [(8, 8), (16, 0), (3, 1), (7, 2)])
@pytest.mark.parametrize("m,n", [(256, 192), (271, 333)])
def test_column_blocks(plan, m, n, pad, lead, dgrad):  # noqa: F811
    """Strided input and output rows, on and off 16-byte alignment; what lies beside the output stays."""
    import torch
    x = bf16((150, m if dgrad else n), 5, pad=pad, lead=lead)
    cols = n if dgrad else m
    wide = torch.full((150, cols + pad), 33.0, dtype=torch.bfloat16, device="cuda")
    w = bf16((3, m, n), 6, 0.1)
    check(plan, x, w, [0, 70, 71, 140], dgrad, out=wide[:, lead:lead + cols])
    assert bool((wide[:, :lead] == 33).all()) and bool((wide[:, lead + cols:] == 33).all())


@pytest.mark.parametrize("dgrad", [False, True])
@pytest.mark.parametrize("shift", [0, 1, 4])
def test_weights_off_alignment(plan, shift, dgrad):  # noqa: F811
    import torch
    flat = bf16((3 * 264 * 136 + 8,), 7, 0.1)
    w = flat[shift:shift + 3 * 264 * 136].view(3, 264, 136)
    check(plan, bf16((90, 264 if dgrad else 136), 8), w, [0, 30, 30, 90], dgrad)


@pytest.mark.parametrize("dgrad", [False, True])
@pytest.mark.parametrize("odd", [False, True])
def test_what_is_not_finite_stays_where_it_is(plan, odd, dgrad):  # noqa: F811
    """NaN rows of one expert, infinities in a weight of another and in the rows behind the last expert reach no
    other expert's rows."""
    import torch
    m, n, edges = (257, 137, [0, 40, 72, 200]) if odd else (256, 136, [0, 40, 72, 200])
    x = bf16((230, m if dgrad else n), 9)
    w = bf16((3, m, n), 10, 0.1)
    x[45] = float("nan")
    x[200:] = float("inf")
    w[2] = float("inf")
    offsets = torch.tensor(edges, dtype=torch.int32, device="cuda")
    out = torch.full((230, n if dgrad else m), 5.0, dtype=torch.bfloat16, device="cuda")
    run(plan, x, w, out, offsets, dgrad)
    plan.sync()
    finite = torch.isfinite(out).all(1)
    want = torch.ones(230, dtype=torch.bool, device="cuda")
    want[45] = False
    want[72:200] = False
    assert torch.equal(finite, want)
    assert bool(torch.isnan(out[45]).all()) and bool((out[200:] == 5).all())


@pytest.mark.parametrize("dgrad", [False, True])
@pytest.mark.parametrize("tokens,m,n", [(1, 512, 8192), (1, 257, 9001), (8, 2048, 4096), (40, 768, 6000), (200, 300, 7000)])
def test_few_tokens_and_long_sums(plan, tokens, m, n, dgrad):  # noqa: F811
    """Sums that are cut into parts and joined."""
    if dgrad:
        m, n = n, m
    w = bf16((m, n), 11, 0.1)
    x = bf16((tokens, m if dgrad else n), 12)
    first = check(plan, x, w, None, dgrad)
    for _ in range(3):
        assert (check(plan, x, w, None, dgrad) == first).all()


@pytest.mark.parametrize("groups", [300, 4096])
@pytest.mark.parametrize("dgrad", [False, True])
def test_many_experts(plan, groups, dgrad):  # noqa: F811
    rng = np.random.default_rng(groups)
    edges = np.concatenate([[0], np.cumsum(rng.integers(0, 3, groups))]).tolist()
    tokens = edges[-1] + 5
    check(plan, bf16((tokens, 72 if dgrad else 40), 13), bf16((groups, 72, 40), 14, 0.1), edges, dgrad)


@pytest.mark.parametrize("dgrad", [False, True])
def test_ragged_experts_of_many_tiles(plan, dgrad):  # noqa: F811
    """More tiles than one turn of the GPU, tiles of every height."""
    rng = np.random.default_rng(5)
    edges = np.concatenate([[0], np.cumsum(rng.integers(0, 700, 24))]).tolist()
    tokens = edges[-1] + 100
    check(plan, bf16((tokens, 1032 if dgrad else 520), 15), bf16((24, 1032, 520), 16, 0.1), edges, dgrad)


@pytest.mark.parametrize("dgrad", [False, True])
def test_one_weight_of_many_turns(plan, dgrad):  # noqa: F811
    check(plan, bf16((9000, 4104 if dgrad else 264), 17), bf16((4104, 264), 18, 0.1), None, dgrad)


@pytest.mark.parametrize("dgrad", [False, True])
@pytest.mark.parametrize("groups", [0, 7, 600])
def test_more_turns_than_are_decoded_at_the_start(plan, groups, dgrad):  # noqa: F811
    """Short sums and thousands of tiles: one weight, a few experts, and more experts than have a place each."""
    rng = np.random.default_rng(9)
    if groups == 600:
        edges = np.concatenate([[0], np.cumsum(rng.integers(0, 90, groups))]).tolist()
        m, n = 3600, 16
    else:
        edges = [0] + np.sort(rng.integers(0, 100000, max(groups, 1) - 1)).tolist() + [100000]
        m, n = 6000, 8
    if dgrad:
        m, n = n, m
    w = bf16((groups, m, n) if groups else (m, n), 30)
    check(plan, bf16((edges[-1], m if dgrad else n), 31), w, edges if groups else None, dgrad)


@pytest.mark.parametrize("dgrad", [False, True])
def test_weights_beyond_2_31_values(plan, dgrad):  # noqa: F811
    import torch
    m, n, groups = 8192, 16384, 17
    w = torch.zeros((groups, m, n), dtype=torch.bfloat16, device="cuda")
    w[16].normal_()
    w[1].normal_()
    check(plan, bf16((40, m if dgrad else n), 19, 0.1), w, [0, 0, 10] + [10] * 14 + [40], dgrad)


@pytest.mark.parametrize("dgrad", [False, True])
@pytest.mark.parametrize("tokens,m,n,groups", [(36000, 521, 4001, 0), (40, 16001, 8193, 0), (16100, 8193, 4097, 0),
                                               (700, 2501, 3001, 24), (36000, 264, 4000, 0)])
def test_rows_that_are_not_aligned_in_chunks(plan, tokens, m, n, groups, dgrad):  # noqa: F811
    """Operands that do not fit the room for aligned rows at once: chunks of tokens, of experts and of outputs."""
    rng = np.random.default_rng(7)
    x = bf16((tokens, m if dgrad else n), 28, pad=1)      # an odd pitch whatever the width
    w = bf16((groups, m, n) if groups else (m, n), 29, 0.1)
    edges = None
    if groups:
        edges = [3] + (3 + np.sort(rng.integers(0, tokens - 9, groups - 1))).tolist() + [tokens - 4]
        edges[5] = edges[6]                                # an expert without tokens
    check(plan, x, w, edges, dgrad)


def test_no_tokens(plan):  # noqa: F811
    import torch
    x, out = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), torch.empty((0, 32), dtype=torch.bfloat16, device="cuda")
    plan.product(x, bf16((32, 64), 1), out)
    plan.product(x, bf16((2, 32, 64), 1), out, offsets=torch.zeros(3, dtype=torch.int32, device="cuda"))
    full = torch.full((9, 32), 4.0, dtype=torch.bfloat16, device="cuda")
    plan.product(bf16((9, 64), 2), bf16((2, 32, 64), 1), full, offsets=torch.zeros(3, dtype=torch.int32, device="cuda"))
    plan.sync()
    assert bool((full == 4).all())


@pytest.mark.parametrize("m,n", [(512, 256), (333, 215)])
def test_on_another_stream_and_captured(plan, m, n):  # noqa: F811
    """A captured call sees what its tensors hold at each replay, the offsets among it."""
    import torch
    x, w = bf16((400, n), 20), bf16((4, m, n), 21, 0.1)
    edges = [[0, 100, 200, 300, 400], [0, 0, 390, 395, 399], [0, 0, 0, 0, 0]]
    offsets = torch.tensor(edges[0], dtype=torch.int32, device="cuda")
    y = torch.zeros((400, m), dtype=torch.bfloat16, device="cuda")
    dx = torch.zeros((400, n), dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    plan.product(x, w, y, offsets=offsets, stream=s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.product(x, w, y, offsets=offsets)
        plan.dgrad(y, w, dx, offsets=offsets)
    for e in edges:
        offsets.copy_(torch.tensor(e, dtype=torch.int32))
        x.copy_(bf16((400, n), 22))
        y.zero_(), dx.zero_()
        graph.replay()
        y2, dx2 = torch.zeros_like(y), torch.zeros_like(dx)
        check(plan, x, w, e, False, out=y2)
        check(plan, y2, w, e, True, out=dx2)
        assert torch.equal(y, y2) and torch.equal(dx, dx2)
    plan.sync()


def test_the_three_products_agree_with_differences(mu, plan):  # noqa: F811
    """L = sum(dy * y): dx and the weight gradient against L's change along a direction, in fp64 from the bf16
    results' own bounds: y is linear in x and W, so the differences are exact."""
    import torch
    edges, m, n = [0, 33, 33, 90], 264, 136
    offsets = torch.tensor(edges, dtype=torch.int32, device="cuda")
    x, w, dy = bf16((90, n), 23), bf16((3, m, n), 24, 0.1), bf16((90, m), 25)
    x8 = mu.Act8.empty(90, n, "int8")
    mu.act_pack(x, x8)
    mu.act_unpack(x8, x)
    dx = torch.empty_like(x)
    dw = torch.empty((3, m, n), device="cuda")
    plan.dgrad(dy, w, dx, offsets=offsets)
    plan.wgrad(dy, x8, dw, offsets=offsets)
    plan.sync()

    def loss(a, b):
        return sum(float((dy[p:q].double() * (a[p:q] @ b[e].t())).sum()) for e, p, q in ranges(edges, 90))
    vx, vw = bf16((90, n), 26).double(), bf16((3, m, n), 27).double()
    x64, w64 = x.double(), w.double()
    along_x = loss(x64 + vx, w64) - loss(x64, w64)
    along_w = loss(x64, w64 + vw) - loss(x64, w64)
    size_x = sum(float((vx[p:q].abs() * (dy[p:q].double().abs() @ w64[e].abs())).sum()) for e, p, q in ranges(edges, 90))
    size_w = sum(float((vw[e].abs() * (dy[p:q].double().abs().t() @ x64[p:q].abs())).sum()) for e, p, q in ranges(edges, 90))
    # dx: (2 m + 8) u of its terms and a bf16 rounding (2^-8 of the result, which the terms bound); fp64 of loss
    assert abs(float((dx.double() * vx).sum()) - along_x) <= ((2 * m + 8) * U + 2.0 ** -8 + 1e-10) * size_x
    assert abs(float((dw.double() * vw).sum()) - along_w) <= ((2 * 90 + 8) * U + 1e-10) * size_w


def test_what_the_binding_refuses(mu, plan):  # noqa: F811
    import torch
    x, w, y = bf16((8, 40), 1), bf16((3, 24, 40), 2), bf16((8, 24), 3)
    o = torch.tensor([0, 2, 5, 8], dtype=torch.int32, device="cuda")
    bad = [lambda: plan.product(x.float(), w, y, offsets=o), lambda: plan.product(x, w.float(), y, offsets=o),
           lambda: plan.product(x, w, y.float(), offsets=o), lambda: plan.product(x, w, y, offsets=o.long()),
           lambda: plan.product(x, w, y, offsets=o[:3]), lambda: plan.product(x, w, y, offsets=o[:1]),
           lambda: plan.product(x, w, y), lambda: plan.product(x, w[0], y, offsets=o), lambda: plan.product(x, w[0], x),
           lambda: plan.product(x, w.transpose(1, 2), y, offsets=o), lambda: plan.product(x[:, :39], w, y, offsets=o),
           lambda: plan.product(x[:7], w, y, offsets=o), lambda: plan.dgrad(x, w, y, offsets=o),
           lambda: plan.product(x.cpu(), w, y, offsets=o), lambda: plan.product(x, w.cpu(), y, offsets=o),
           lambda: plan.product(x.t(), w, y, offsets=o)]
    for call in bad:
        with pytest.raises(ValueError):
            call()
    square = bf16((40, 40), 4)
    with pytest.raises(mu.MuonError):
        plan.product(x, square, x)                       # in place

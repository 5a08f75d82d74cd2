"""Calls of the experts' operators at their limits, on the GPU."""
import numpy as np
import pytest

from test_gpu_experts import on_gpu, order, ordered, routed
from test_gpu_layer import U, mu, plan, rand  # noqa: F401  (fixtures)
from test_gpu_product import bf16, check, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("with_drows", [False, True])
def test_gradient_of_the_weights_needs_the_rows(mu, with_drows):  # noqa: F811
    """Without rows the call is refused and writes nothing; every operand has memory of its own."""
    import torch
    slots, n = routed(8, 2, 0)
    dout, w, dw = rand((8, 40), "f32", 1), torch.rand((8, 2), device="cuda"), torch.full((8, 2), 3.0, device="cuda")
    drows = torch.full((n, 40), 5.0, device="cuda") if with_drows else None
    with pytest.raises(mu.MuonError):
        mu.expert_combine_backward(dout, on_gpu(slots), w, drows=drows, dweights=dw)
    torch.cuda.synchronize()
    assert bool((dw == 3).all()) and (drows is None or bool((drows == 5).all()))


def test_gradient_of_the_weights_among_no_rows(mu):  # noqa: F811
    """A tensor of no rows is given, not missing: no slot names a row, every gradient is zero."""
    import torch
    slots, _ = routed(8, 2, 0)
    dw = torch.full((8, 2), 3.0, device="cuda")
    mu.expert_combine_backward(rand((8, 40), "f32", 1), on_gpu(slots), torch.rand((8, 2), device="cuda"),
                               rows=torch.empty((0, 40), device="cuda"), dweights=dw)
    assert bool((dw == 0).all())


@pytest.mark.parametrize("dgrad", [False, True])
@pytest.mark.parametrize("tokens,m,n,groups", [(16, 1024, 8192, 0), (256, 512, 6000, 0), (24, 512, 4096, 3)])
def test_joined_parts_are_this_calls(plan, tokens, m, n, groups, dgrad):  # noqa: F811
    """Sums that are cut into parts, call after call with inputs that take turns: the parts that a call joins are its
    own, not the ones that the workspace held before."""
    import torch
    if dgrad:
        m, n = n, m
    w = bf16((groups, m, n) if groups else (m, n), 1, 0.1)
    edges = [i * tokens // groups for i in range(groups + 1)] if groups else None
    xs = [bf16((tokens, m if dgrad else n), 2 + i) for i in range(2)]
    want = [check(plan, x, w, edges, dgrad) for x in xs]
    offsets = None if edges is None else torch.tensor(edges, dtype=torch.int32, device="cuda")
    out = torch.empty_like(want[0])
    same = torch.ones((), dtype=torch.bool, device="cuda")
    for i in range(100):
        run(plan, xs[i & 1], w, out, offsets, dgrad)
        same &= (out == want[i & 1]).all()
    plan.sync()
    assert bool(same)


@pytest.fixture(scope="module")
def least(mu):  # noqa: F811
    """A plan without bytes for copies alone."""
    with mu.GradPlan(aligned_bytes=0) as p:
        yield p
        p.sync()


@pytest.mark.parametrize("dgrad", [False, True])
@pytest.mark.parametrize("tokens,m,n,groups", [(33, 257, 129, 0), (4000, 521, 4001, 0), (40, 6001, 8193, 0),
                                               (5001, 2049, 4097, 0), (700, 1001, 2001, 24), (9000, 264, 4000, 0)])
def test_copies_in_the_shared_room(least, tokens, m, n, groups, dgrad):  # noqa: F811
    """Unaligned rows on the smallest plan, in one piece and in many."""
    x = bf16((tokens, m if dgrad else n), 28, pad=1)
    w = bf16((groups, m, n) if groups else (m, n), 29, 0.1)
    edges = [3] + [3 + (tokens - 9) * i * i // (groups * groups) for i in range(1, groups)] + [tokens - 4] if groups else None
    check(least, x, w, edges, dgrad)


def test_the_shared_room_between_other_calls(mu, least):  # noqa: F811
    """Copies lie where the weight gradient keeps partial sums and the norm its own: each call finds what it needs."""
    import torch
    dy, x = bf16((9000, 512), 1), bf16((9000, 264), 2)
    x8, dw = mu.Act8.empty(9000, 264, "int8"), [torch.empty((512, 264), device="cuda") for _ in range(2)]
    mu.act_pack(x, x8)
    mu.act_unpack(x8, x)
    norm = [torch.zeros(1, device="cuda") for _ in range(2)]
    odd, w = bf16((5000, 1001), 3), bf16((4001, 1001), 4, 0.1)
    out = [torch.empty((5000, 4001), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    for i in range(2):
        least.wgrad(dy, x8, dw[i])
        least.product(odd, w, out[i])
        least.grad_norm([dw[i]], norm[i])
    least.sync()
    assert torch.equal(*dw) and torch.equal(*out) and torch.equal(*norm)
    want, size = dy.double().t() @ x.double(), dy.double().abs().t() @ x.double().abs()
    assert bool(((dw[0].double() - want).abs() <= (2 * 9000 + 8) * U * size).all())
    check(least, odd, w, None, False)


@pytest.mark.parametrize("dgrad", [False, True])
def test_rows_that_no_piece_holds(mu, plan, least, dgrad):  # noqa: F811
    """64 rows of 2^20 - 1 values: refused on the smallest plan with nothing written, computed on the usual one."""
    import torch
    m, n, tokens = 70, (1 << 20) - 1, 65
    w = bf16((m, n), 5, 0.01)
    if dgrad:
        w = w.t().contiguous()
    x, out = bf16((tokens, n), 6), torch.full((tokens, m), 7.0, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(mu.MuonError) as refused:
        run(least, x, w, out, None, dgrad)
    assert refused.value.code == mu.MUON_ERR_UNSUPPORTED
    least.sync()
    assert bool((out == 7).all())
    check(plan, x, w, None, dgrad)


@pytest.mark.parametrize("choices,experts", [(1, 64), (3, 64), (4, 300), (8, 512), (5, 1023), (4, 1024), (7, 1025)])
def test_order_of_long_lists(mu, choices, experts):  # noqa: F811
    """Lists just below and at the length from which the largest clusters are taken, and a million ids."""
    rng = np.random.default_rng(experts + choices)
    edge = -(-256 * (experts + 128) // choices)
    for tokens in (edge - 1, edge, (1 << 20) // choices):
        ids = rng.integers(-1, experts + 1, (tokens, choices))
        offsets, slots = ordered(mu, ids, experts)
        want = order(ids, experts)
        assert np.array_equal(offsets.cpu().numpy(), want[0]) and np.array_equal(slots.cpu().numpy(), want[1])


@pytest.mark.parametrize("tokens,m,n,groups", [(20000, 521, 392, 0), (12000, 264, 1032, 6)])
def test_weight_gradient_of_copied_rows_over_many_rounds(mu, plan, tokens, m, n, groups):  # noqa: F811
    """dy off 16-byte alignment, hundreds of rounds of the operands' ring, call after call: none gives up a wait, and all
    give the same bits."""
    import torch
    dy, x = bf16((tokens, m), 1, 0.5, pad=1), bf16((tokens, n), 2)
    x8 = mu.Act8.empty(tokens, n, "e4m3")
    mu.act_pack(x, x8)
    mu.act_unpack(x8, x)
    edges = [tokens * i * i // (groups * groups) for i in range(groups + 1)] if groups else [0, tokens]
    offsets = torch.tensor(edges, dtype=torch.int32, device="cuda") if groups else None
    g = [torch.empty((groups, m, n) if groups else (m, n), device="cuda") for _ in range(2)]
    same = torch.ones((), dtype=torch.bool, device="cuda")
    for i in range(40):
        plan.wgrad(dy, x8, g[i > 0], offsets=offsets)
        same &= (g[i > 0] == g[0]).all()
    plan.sync()                                   # raises where a wait ran out
    assert bool(same)
    for e, (a, b) in enumerate(zip(edges, edges[1:])):
        d, v = dy[a:b].double().t(), x[a:b].double()
        got = (g[0][e] if groups else g[0]).double()
        assert bool(((got - d @ v).abs() <= (2 * (b - a) + 8) * U * (d.abs() @ v.abs())).all())

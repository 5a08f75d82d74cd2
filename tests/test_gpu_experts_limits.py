"""Calls of the experts' operators at their limits, on the GPU."""
import pytest

from test_gpu_experts import on_gpu, routed
from test_gpu_layer import mu, plan, rand  # noqa: F401  (fixtures)
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

"""Calls of the gradient norm and clipping at their limits, on the GPU."""
import numpy as np
import pytest

from test_gpu_layer import U, dt, mu, plan  # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("at", [0, 57, 99])
def test_norm_does_not_lie_in_a_gradient(mu, plan, at):  # noqa: F811
    """Refused, and the gradients stay as they are; beside them it may lie."""
    import torch
    both = torch.full((101,), 2.0, device="cuda")
    with pytest.raises(mu.MuonError):
        plan.grad_norm([both[:100]], both[at:at + 1])
    torch.cuda.synchronize()
    assert bool((both == 2).all())
    plan.grad_norm([both[:100]], both[100:])
    assert float(both[100]) == 20.0 and bool((both[:100] == 2).all())


def laid_out(sizes, dtypes, gaps, fill):
    """One buffer per type, filled, and in it a tensor of each size, `gaps` values apart."""
    import torch
    ends = {d: 0 for d in ("f32", "bf16")}
    for n, d, gap in zip(sizes, dtypes, gaps):
        ends[d] += gap + n
    buffers = {d: torch.full((n + 16,), fill, dtype=dt(d), device="cuda") for d, n in ends.items()}
    return buffers, list(views(buffers, sizes, dtypes, gaps))


def views(buffers, sizes, dtypes, gaps):
    at = {d: 0 for d in buffers}
    for n, d, gap in zip(sizes, dtypes, gaps):
        at[d] += gap
        yield buffers[d][at[d]:at[d] + n]
        at[d] += n


@pytest.mark.parametrize("kinds", ["in place", "same", "other", "bf16", "f32"])
@pytest.mark.parametrize("count", [30, 100, 960, 961, 2600])
def test_lists_of_any_length(mu, plan, count, kinds):  # noqa: F811
    """Every value of long lists, over every table's length: gradients of both types at any offset, some empty, some of
    many chunks.  The factor is one fp32 division, a value one fp32 product and one rounding, as torch's are: equal bits.
    What lies between the tensors stays."""
    import torch
    rng = np.random.default_rng(count)
    sizes = np.exp(rng.uniform(0, 7, count)).astype(int)
    sizes[rng.random(count) < 0.05] = 0
    sizes[rng.choice(count, 3, replace=False)] = rng.integers(20000, 70000, 3)
    sizes = [int(v) for v in sizes]
    dtypes = [("f32", "bf16")[i] for i in rng.integers(0, 2, count)]
    gaps = [int(v) for v in rng.integers(0, 9, count)]
    buffers, grads = laid_out(sizes, dtypes, gaps, 3.0)
    g = torch.Generator(device="cuda").manual_seed(count)
    for t in grads:
        t.copy_(torch.randn(t.shape, generator=g, device="cuda") * 0.01)
    before = {d: b.clone() for d, b in buffers.items()}
    norm = torch.zeros(1, device="cuda")
    plan.grad_norm(grads, norm)
    want = float(np.sqrt(sum(float((t.double() ** 2).sum()) for t in grads)))
    assert abs(float(norm) - want) <= 18 * U * want
    factor = torch.tensor([want / 2], device="cuda")   # a largest norm that is exact in fp32
    most = float(factor)
    factor = factor / norm
    if kinds == "in place":
        plan.grad_clip(grads, norm, most)
        expected = before
        for d, t in zip(dtypes, views(expected, sizes, dtypes, gaps)):
            t.copy_((t.float() * factor).to(dt(d)))
        assert all(torch.equal(buffers[d], expected[d]) for d in buffers)
        return
    types = {"same": dtypes, "other": [{"f32": "bf16", "bf16": "f32"}[d] for d in dtypes]}.get(kinds, [kinds] * count)
    shifted = [int(v) for v in rng.integers(0, 9, count)]
    results, out = laid_out(sizes, types, shifted, 5.0)
    expected = {d: b.clone() for d, b in results.items()}
    plan.grad_clip(grads, norm, most, out=out)
    for d, t, x in zip(types, views(expected, sizes, types, shifted), grads):
        t.copy_((x.float() * factor).to(dt(d)))
    assert all(torch.equal(results[d], expected[d]) for d in results)
    assert all(torch.equal(buffers[d], before[d]) for d in buffers)

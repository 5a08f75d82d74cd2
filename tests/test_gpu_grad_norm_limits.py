"""Calls of the gradient norm and clipping at their limits, on the GPU."""
import pytest

from test_gpu_layer import mu, plan  # noqa: F401  (fixtures)

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

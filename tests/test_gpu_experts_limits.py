"""Calls of the experts' operators at their limits, on the GPU."""
import pytest

from test_gpu_experts import on_gpu, routed
from test_gpu_layer import mu, rand  # noqa: F401  (fixture)

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

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

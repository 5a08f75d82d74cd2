"""examples/train_ffn.py: the layer-side operators and the Muon step together."""
import importlib.util
import os

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location("train_ffn", os.path.join(ROOT, "examples", "train_ffn.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_gradients_follow_from_what_was_saved(ex, fmt):
    """Each gradient against its formula in 64 bits on the 8-bit copies and bf16 tensors that the block
    holds, within the bounds of fp32 sums (see test_gpu_layer) and the bf16 roundings of their ends."""
    import torch
    from oracle import layer_ref as L
    from test_gpu_layer import U, close, f64, values
    t, h, f = 512, 256, 640
    b = ex.FFNBlock(t, h, f, fmt)
    x, dy = (torch.randn((t, h), device="cuda", generator=torch.Generator(device="cuda").manual_seed(k)).bfloat16()
             for k in (5, 6))
    b.gain.copy_(1 + 0.2 * torch.randn(h, device="cuda", generator=torch.Generator(device="cuda").manual_seed(7)))
    b.forward(x)
    dx = b.backward(dy)
    dn = b.dgu @ b.low[0]          # the product that backward() formed
    b.sync()
    for grad, d, v, s in ((b.grads[1], f64(dy), values(b.a8), 1.0), (b.grads[0], f64(b.dgu), values(b.norm8), f64(b.gain))):
        close(grad, d.T @ v * s, 2 * (t + 16) * U * (np.abs(d).T @ np.abs(v)) * np.abs(s))
    n, w = values(b.norm8), f64(b.gain)
    want, dgain = L.rmsnorm_grad(f64(dn), n, f64(b.rstd), w, f64(dy))
    k = np.abs(f64(dn) * w)
    r = f64(b.rstd)[:, None]
    close(dx, want, U * (r * (6 * k + 110 * np.abs(n) * np.mean(k * np.abs(n), 1, keepdims=True)) + 2 * np.abs(f64(dy))
                         + 2 * np.abs(want)))
    close(b.dgain, dgain, U * (t + 20) * np.sum(np.abs(f64(dn) * n), 0))


def test_training_reduces_the_loss(ex):
    losses, block = ex.train(tokens=1024, hidden=256, ffn=640, steps=12)
    assert all(b < a for a, b in zip(losses, losses[1:]))
    assert block.saved_bytes() < 0.55 * 1024 * (2 * 2 * 256 + 3 * 2 * 640)

"""examples/train_moe.py: the order of tokens, the moves, the three products by expert, the activation, the norm,
the clipping and the optimizer step as a block of experts uses them."""
import importlib.util
import os

import numpy as np
import pytest

from test_gpu_experts import order
from test_gpu_layer import U, close, f64, values
from test_gpu_product import rounded

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SIZES = [(512, 256, 128, 8, 2), (301, 261, 139, 11, 3), (1, 128, 64, 4, 4)]


@pytest.fixture(scope="module")
def ex():
    torch = pytest.importorskip("torch")
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    spec = importlib.util.spec_from_file_location("train_moe", os.path.join(ROOT, "examples", "train_moe.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def gauss(shape, seed, scale=1.0):
    import torch
    return (torch.randn(shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)) * scale).bfloat16()


def check_product(got, x, w, edges, transposed):
    for e, (a, b) in enumerate(zip(edges, edges[1:])):
        if a < b:
            we = w[e].double() if transposed else w[e].double().t()
            want, size = x[a:b].double() @ we, x[a:b].double().abs() @ we.abs()
            bound = (2 * x.shape[1] + 8) * U * size
            y = got[a:b].double()
            assert bool(((rounded(want - bound) <= y) & (y <= rounded(want + bound))).all())


@pytest.mark.parametrize("tokens,hidden,ffn,experts,choices", SIZES)
def test_each_stage_follows_from_the_one_before(ex, tokens, hidden, ffn, experts, choices):
    """Every operator's outputs in the run of the block, within its bounds on the inputs that the run handed it."""
    import torch
    b = ex.MoEBlock(tokens, hidden, ffn, experts, choices)
    x, dy = gauss((tokens, hidden), 5), gauss((tokens, hidden), 6)
    b.forward(x)
    b.backward(dy)
    b.sync()
    offsets, slots = order(b.ids.cpu().numpy(), experts)
    assert np.array_equal(b.offsets.cpu().numpy(), offsets) and np.array_equal(b.slots.cpu().numpy(), slots)
    token = np.empty(tokens * choices, int)
    token[slots.reshape(-1)] = np.arange(tokens * choices) // choices
    assert torch.equal(b.xs, x[torch.tensor(token, device="cuda")])
    check_product(b.gu, b.xs, b.low[0], offsets, False)
    check_product(b.ys, b.a, b.low[1], offsets, False)
    p = f64(b.weights_of)[:, :, None]
    terms = p * f64(b.ys)[slots]
    close(b.y, terms.sum(1), (choices + 1) * U * np.abs(terms).sum(1))
    terms = f64(dy)[:, None, :] * f64(b.ys)[slots]
    close(b.dp, terms.sum(2), (hidden + 8) * U * np.abs(terms).sum(2))
    want = np.empty((tokens * choices, hidden))
    want[slots.reshape(-1)] = (p * f64(dy)[:, None, :]).reshape(-1, hidden)
    close(b.dys, want, U * np.abs(want))
    check_product(b.da, b.dys, b.low[1], offsets, True)
    check_product(b.dxs, b.dgu, b.low[0], offsets, True)
    for grad, d, v in ((b.sums[1], f64(b.dys), values(b.a8)), (b.sums[0], f64(b.dgu), values(b.x8))):
        for e in range(experts):
            r = slice(offsets[e], offsets[e + 1])
            size = np.abs(d[r]).T @ np.abs(v[r])
            # fp32 gradients below 2^-126 become zero
            close(grad[e], d[r].T @ v[r], 2 * (r.stop - r.start + 16) * U * size + 2.0 ** -126)
    terms = f64(b.dxs)[slots]
    close(b.dx, terms.sum(1), (choices + 1) * U * np.abs(terms).sum(1))


@pytest.mark.parametrize("tokens,hidden,ffn,experts,choices", SIZES[:2])
def test_gradients_of_the_block(ex, tokens, hidden, ffn, experts, choices):
    """Against the gradients of the block's formula in 64 bits, by automatic differentiation.  On the way to any of
    them lie at most eight bf16 roundings (each at most 2^-8 of its value) and two to 8 bits (half a step of
    1/127 of a group's largest value, about 2.5 times its root mean square: 1 % of it): 8 * 0.4 % + 2 * 1 % < 6 %."""
    import torch
    b = ex.MoEBlock(tokens, hidden, ffn, experts, choices)
    x, dy = gauss((tokens, hidden), 5), gauss((tokens, hidden), 6)
    y = b.forward(x)
    dx = b.backward(dy)
    b.sync()
    x64 = x.double().requires_grad_()
    wr, wgu, wd = (t.double().requires_grad_() for t in (b.router, b.low[0], b.low[1]))
    prob = torch.softmax(x64 @ wr.t(), 1)
    out = x64
    for j in range(choices):
        e = b.ids[:, j].long()
        gu = torch.einsum("th,tfh->tf", x64, wgu[e])
        a = torch.nn.functional.silu(gu[:, :ffn]) * gu[:, ffn:]
        out = out + prob.gather(1, e[:, None]) * torch.einsum("tf,thf->th", a, wd[e])
    out.backward(dy.double())
    for got, want in ((y, out), (dx, x64.grad), (b.sums[0], wgu.grad), (b.sums[1], wd.grad), (b.drouter, wr.grad)):
        want = want.detach()
        assert float((got.double() - want).norm()) <= 0.06 * float(want.norm())


def test_clipped_step(ex):
    """The step reads the fp32 sums scaled to the largest norm: the same weights as from gradients scaled by hand."""
    import torch
    import matrix_orthogonalising_optimizer_muon_gb300 as muon
    t, h, f, experts, k = 256, 136, 72, 6, 2
    b = ex.MoEBlock(t, h, f, experts, k)
    b.forward(gauss((t, h), 5))
    b.backward(gauss((t, h), 6))
    b.sync()
    sums, router, drouter = [s.clone() for s in b.sums], b.router.clone(), b.drouter.clone()
    want = [[w.clone() for w in ws] for ws in b.weights]
    total = np.sqrt(sum(float((s.double() ** 2).sum()) for s in sums + [drouter]))
    largest = total / 3
    b.step(1e-2, max_norm=largest)
    b.sync()
    assert abs(float(b.norm) - total) <= 18 * U * total
    factor = torch.tensor(largest, device="cuda") / b.norm
    grads = [(s * factor).bfloat16() for s in sums]
    assert all(torch.equal(a, c) for a, c in zip(grads, b.grads))
    flat = [w for ws in want for w in ws]
    momentum = [torch.zeros_like(w) for w in flat]
    with muon.MuonPlan([tuple(w.shape) for w in flat], "bf16") as p:
        p.step(flat, [g for gs in grads for g in gs], momentum, 1e-2, 0.0)
        p.sync()
    assert all(torch.equal(a, c) for a, c in zip(flat, [w for ws in b.weights for w in ws]))
    assert torch.equal(b.router, router - 1e-2 * (drouter * factor))


def test_captured_passes(ex):
    """Both passes in one graph: replayed on other tokens they give the bits of the eager calls."""
    import torch
    t, h, f, experts, k = 320, 136, 72, 6, 2
    b, c = (ex.MoEBlock(t, h, f, experts, k) for _ in range(2))
    x, dy = gauss((t, h), 5), gauss((t, h), 6)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):
            b.forward(x)
            b.backward(dy)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = b.forward(x)
        dx = b.backward(dy)
        b.grad_plan.grad_norm(b.clip_in, b.norm)
    for seed in (7, 8):
        x.copy_(gauss((t, h), seed)), dy.copy_(gauss((t, h), seed + 10))
        for m in (b, c):
            for g in m.sums + [m.drouter]:
                g.zero_()
        graph.replay()
        y2 = c.forward(x)
        dx2 = c.backward(dy)
        c.grad_plan.grad_norm(c.clip_in, c.norm)
        torch.cuda.synchronize()
        assert torch.equal(y, y2) and torch.equal(dx, dx2) and torch.equal(b.norm, c.norm)
        assert all(torch.equal(p, q) for p, q in zip(b.sums, c.sums))
    b.sync(), c.sync()


def test_the_example_runs(ex):
    losses, norms, _ = ex.train(tokens=512, hidden=128, ffn=72, experts=6, choices=2, steps=4)
    assert len(losses) == 4 and all(np.isfinite(losses)) and all(n > 0 for n in norms)

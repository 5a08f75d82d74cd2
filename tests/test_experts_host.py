"""Refusals of the experts' and gradient-norm entry points, on the CPU: every bad argument is reported before any
CUDA call, as a status code by the C functions and as ValueError by the binding."""
import ctypes

import pytest

import matrix_orthogonalising_optimizer_muon_gb300 as mu

torch = pytest.importorskip("torch")
A, B, C, D, E, F = (0x100000000 * k for k in range(1, 7))   # far apart, 16-byte aligned, never dereferenced
BAD, UNSUP = mu.MUON_ERR_INVALID_ARG, mu.MUON_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    return mu.load()


def handle():
    """A grad plan's handle that is never read: bad arguments are found first."""
    return ctypes.cast(ctypes.create_string_buffer(256), ctypes.c_void_p)


@pytest.mark.parametrize("name", ["muon_product", "muon_dgrad"])
@pytest.mark.parametrize("kw,code", [
    (dict(plan=None), BAD), (dict(x=None), BAD), (dict(w=None), BAD), (dict(y=None), BAD), (dict(tokens=-1), BAD),
    (dict(tokens=1 << 31), UNSUP), (dict(tokens=(1 << 31) - 4095), UNSUP), (dict(m=0), BAD), (dict(n=0), BAD), (dict(m=(1 << 20) + 1, ld=1 << 21), UNSUP),
    (dict(n=(1 << 20) + 1, ld=1 << 21), UNSUP), (dict(ldx=49), BAD), (dict(ldy=49), BAD), (dict(x=A + 1), BAD),
    (dict(y=C + 1), BAD), (dict(w=B + 1), BAD), (dict(groups=-1), BAD), (dict(groups=4097, offsets=D), BAD),
    (dict(groups=2), BAD), (dict(offsets=D), BAD), (dict(offsets=D + 2, groups=2), BAD), (dict(y=A), BAD),
    (dict(y=B), BAD), (dict(y=B + 50 * 50 * 2 * 2 - 2, groups=2, offsets=D), BAD), (dict(y=D, groups=2, offsets=D), BAD),
    (dict(ldx=1 << 31), BAD), (dict(ldy=1 << 31), BAD)])
def test_products_refuse(lib, name, kw, code):
    a = dict(plan=handle(), x=A, w=B, y=C, tokens=4, m=50, n=50, offsets=None, groups=0, ld=50)
    a.update(kw)
    ldx, ldy = a.get("ldx", a["ld"]), a.get("ldy", a["ld"])
    assert getattr(lib, name)(a["plan"], a["x"], ldx, a["w"], a["tokens"], a["m"], a["n"], a["offsets"], a["groups"],
                              a["y"], ldy, None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(ids=None), BAD), (dict(offsets=None), BAD), (dict(slots=None), BAD), (dict(tokens=-1), BAD),
    (dict(choices=0), BAD), (dict(choices=65), BAD), (dict(experts=0), BAD), (dict(experts=4097), BAD),
    (dict(tokens=1 << 30, choices=2), UNSUP), (dict(ids=A + 2), BAD), (dict(slots=A), BAD), (dict(offsets=A + 4), BAD),
    (dict(offsets=C), BAD), (dict(tokens=1 << 31), UNSUP)])
def test_order_refuses(lib, kw, code):
    a = dict(ids=A, tokens=10, choices=2, experts=8, offsets=B, slots=C)
    a.update(kw)
    assert lib.muon_expert_order(a["ids"], a["tokens"], a["choices"], a["experts"], a["offsets"], a["slots"], None) == code


MOVE = dict(tokens=4, choices=2, rows=8, cols=50, dtype=1, ld=50, ldr=50)
MOVES = [(dict(tokens=-1), BAD), (dict(choices=0), BAD), (dict(choices=65), BAD), (dict(rows=-1), BAD), (dict(cols=0), BAD),
         (dict(cols=(1 << 20) + 1), UNSUP), (dict(dtype=2), UNSUP), (dict(rows=1 << 31), UNSUP), (dict(ld=49), BAD),
         (dict(ldr=49), BAD), (dict(slots=None), BAD), (dict(slots=C + 1), BAD), (dict(x=None), BAD), (dict(x=A + 1), BAD),
         (dict(r=B + 1), BAD), (dict(tokens=1 << 30), UNSUP)]


@pytest.mark.parametrize("kw,code", MOVES + [(dict(r=None), BAD), (dict(r=A), BAD), (dict(r=C), BAD), (dict(r=A + 50), BAD)])
def test_dispatch_refuses(lib, kw, code):
    a = dict(MOVE, x=A, r=B, slots=C)
    a.update(kw)
    assert lib.muon_expert_dispatch(a["x"], a["ld"], a["slots"], a["tokens"], a["choices"], a["rows"], a["cols"],
                                    a["dtype"], a["r"], a["ldr"], None) == code


@pytest.mark.parametrize("kw,code", MOVES + [(dict(r=None), BAD), (dict(r=A), BAD), (dict(x=C), BAD), (dict(x=D), BAD),
                                             (dict(w=D + 1), BAD)])
def test_combine_refuses(lib, kw, code):
    a = dict(MOVE, x=A, r=B, slots=C, w=D)
    a.update(kw)
    assert lib.muon_expert_combine(a["r"], a["ldr"], a["slots"], a["w"], a["tokens"], a["choices"], a["rows"], a["cols"],
                                   a["dtype"], a["x"], a["ld"], None) == code


@pytest.mark.parametrize("kw,code", MOVES + [(dict(w=None), BAD), (dict(r=None), BAD), (dict(dr=None, dw=None), BAD),
                                             (dict(dr=A), BAD), (dict(dr=B), BAD), (dict(dw=D), BAD), (dict(dw=C), BAD),
                                             (dict(dr=F, dw=F), BAD), (dict(dr=E + 1), BAD)])
def test_combine_backward_refuses(lib, kw, code):
    a = dict(MOVE, x=A, r=B, slots=C, w=D, dr=E, dw=F)
    a.update(kw)
    assert lib.muon_expert_combine_backward(a["x"], a["ld"], a["slots"], a["w"], a["r"], a["ldr"], a["tokens"],
                                            a["choices"], a["rows"], a["cols"], a["dtype"], a["dr"], a["ldr"], a["dw"],
                                            None) == code


def lists(spec):
    """spec: (pointer, count, dtype) of each -> three ctypes arrays and n."""
    n = len(spec)
    return ((ctypes.c_void_p * n)(*[p for p, _, _ in spec]), (ctypes.c_int64 * n)(*[c for _, c, _ in spec]),
            (ctypes.c_int32 * n)(*[d for _, _, d in spec]), n)


@pytest.mark.parametrize("spec,code", [
    ([(A, 5, 2)], UNSUP), ([(A, -1, 0)], BAD), ([(None, 5, 0)], BAD), ([(A + 2, 5, 0)], BAD), ([(A + 1, 5, 1)], BAD),
    ([(A, 1 << 43, 0), (B, 1, 0)], UNSUP), ([(A, (1 << 43) + 1, 0)], UNSUP)])
def test_lists_are_checked(lib, spec, code):
    p, c, d, n = lists(spec)
    assert lib.muon_grad_norm(handle(), p, c, d, n, F, None) == code
    assert lib.muon_grad_clip(handle(), p, c, d, n, F, 1.0, None, None, None) == code
    good = lists([(C + (k << 20), s[1] if 0 <= s[1] < 100 else 1, 0) for k, s in enumerate(spec)])
    if all(0 <= s[1] < 100 for s in spec):   # the same list as out
        assert lib.muon_grad_clip(handle(), good[0], good[1], good[2], n, F, 1.0, p, d, None) == code


def test_norm_and_clip_refuse(lib):
    p, c, d, n = lists([(A, 100, 0), (B, 100, 1)])
    assert lib.muon_grad_norm(None, p, c, d, n, F, None) == BAD
    assert lib.muon_grad_norm(handle(), p, c, d, n, None, None) == BAD
    assert lib.muon_grad_norm(handle(), p, c, d, n, F + 2, None) == BAD
    assert lib.muon_grad_norm(handle(), p, c, d, -1, F, None) == BAD
    for missing in range(3):
        a = [p, c, d]
        a[missing] = None
        assert lib.muon_grad_norm(handle(), *a, n, F, None) == BAD
    for bad in (0.0, -1.0, float("inf"), float("nan")):
        assert lib.muon_grad_clip(handle(), p, c, d, n, F, bad, None, None, None) == BAD
    assert lib.muon_grad_clip(None, p, c, d, n, F, 1.0, None, None, None) == BAD
    assert lib.muon_grad_clip(handle(), p, c, d, n, None, 1.0, None, None, None) == BAD
    assert lib.muon_grad_clip(handle(), p, c, d, n, F, 1.0, p, None, None) == BAD
    assert lib.muon_grad_clip(handle(), p, c, d, n, F, 1.0, None, d, None) == BAD


@pytest.mark.parametrize("grads,out", [
    ([(A, 100, 0), (A, 100, 0)], None),                                  # the same gradient twice
    ([(A, 100, 0), (A + 396, 100, 0)], None),                            # the last value of one, the first of another
    ([(A, 100, 0), (F, 100, 0)], None),                                  # the norm among them
    ([(A, 100, 0), (B, 100, 0)], [(C, 100, 0), (C + 200, 100, 0)]),      # outputs on one another
    ([(A, 100, 0), (B, 100, 0)], [(B, 100, 0), (C, 100, 0)]),            # an output on another gradient
    ([(A, 100, 0)], [(A, 100, 1)]),                                      # itself, of another type
    ([(A, 100, 0)], [(A + 4, 100, 0)]),                                  # itself, moved
    ([(A, 100, 0)], [(F - 396, 100, 0)])])                               # an output on the norm
def test_clip_refuses_overlap(lib, grads, out):
    p, c, d, n = lists(grads)
    o = lists(out) if out else (None, None, None, 0)
    assert lib.muon_grad_clip(handle(), p, c, d, n, F, 1.0, o[0], o[2], None) == BAD


def test_binding_refuses_tensors_it_cannot_pass():
    x, i = torch.zeros(4, 50), torch.zeros(4, 2, dtype=torch.int32)
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        mu.expert_order(i, torch.zeros(9, dtype=torch.int32), i.clone())     # on the CPU
    with pytest.raises(ValueError):
        mu.expert_dispatch(x, i, torch.zeros(8, 50))
    with pytest.raises(ValueError):
        mu.expert_combine(torch.zeros(8, 50), i, x)
    with pytest.raises(ValueError):
        mu.expert_combine_backward(x, i, torch.ones(4, 2), drows=torch.zeros(8, 50))
    with pytest.raises(ValueError):
        mu.GradList([x])

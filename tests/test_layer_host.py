"""Refusals of the layer-side entry points, on the CPU: every bad argument is reported
before any CUDA call, as a status code by the C functions and as ValueError by the binding."""
import ctypes

import pytest

import matrix_orthogonalising_optimizer_muon_gb300 as mu

torch = pytest.importorskip("torch")
A, B, C, D, E, F = (0x100000000 * k for k in range(1, 7))   # far apart, 16-byte aligned, never dereferenced
BAD, UNSUP = mu.MUON_ERR_INVALID_ARG, mu.MUON_ERR_UNSUPPORTED


def act(codes=E, scales=F, ldq=64, lds=16, fmt=0, reserved=0):
    return ctypes.byref(mu.MuonAct8(codes, scales, ldq, lds, fmt, reserved))


@pytest.fixture(scope="module")
def lib():
    return mu.load()


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), BAD), (dict(rows=-1), BAD), (dict(cols=0), BAD), (dict(ldx=49), BAD), (dict(dtype=2), UNSUP),
    (dict(rows=1 << 31), UNSUP), (dict(cols=(1 << 20) + 1), UNSUP), (dict(out=None), BAD), (dict(x=A + 1), BAD),
    (dict(out=act(codes=None)), BAD), (dict(out=act(codes=E + 8)), BAD), (dict(out=act(ldq=50)), BAD),
    (dict(out=act(ldq=48)), BAD), (dict(out=act(lds=8)), BAD), (dict(out=act(scales=F + 1)), BAD),
    (dict(out=act(fmt=2)), BAD), (dict(out=act(reserved=1)), BAD), (dict(out=act(codes=A)), BAD),
    (dict(out=act(codes=E, scales=E + 32), pack_only=True), BAD)])
def test_pack_refuses(lib, kw, code):
    a = dict(x=A, rows=4, cols=50, ldx=50, dtype=0, out=act())
    a.update(kw)
    assert lib.muon_act_pack(a["x"], a["rows"], a["cols"], a["ldx"], a["dtype"], a["out"], None) == code
    if not kw.get("pack_only"):   # inputs may overlap one another
        assert lib.muon_act_unpack(a["out"], a["rows"], a["cols"], a["x"], a["ldx"], a["dtype"], None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), BAD), (dict(weight=None), BAD), (dict(eps=0.0), BAD), (dict(eps=float("nan")), BAD),
    (dict(eps=float("inf")), BAD), (dict(cols=32769, ld=32769), UNSUP), (dict(h=None, y=None, saved=None, rstd=None), BAD),
    (dict(y=B), BAD), (dict(h=A + 2), BAD), (dict(rstd=C), BAD), (dict(ld=49), BAD), (dict(weight=A + 2), BAD),
    (dict(y=A, h=A), BAD), (dict(saved=act(codes=A)), BAD)])
def test_rmsnorm_forward_refuses(lib, kw, code):
    a = dict(x=A, residual=B, weight=C, rows=4, cols=50, ld=50, dtype=1, eps=1e-6, h=D, y=D + 4096, saved=act(),
             rstd=D + 8192)
    a.update(kw)
    assert lib.muon_rmsnorm_forward(a["x"], a["ld"], a["residual"], a["ld"], a["weight"], a["rows"], a["cols"],
                                    a["dtype"], a["eps"], a["h"], a["ld"], a["y"], a["ld"], a["saved"], 0, a["rstd"],
                                    None) == code


@pytest.mark.parametrize("kw", [dict(gate=None), dict(up=None), dict(a=None, saved=None), dict(a=A + 64), dict(ld=49),
                                dict(saved=act(codes=B))])
def test_swiglu_forward_refuses(lib, kw):
    a = dict(gate=A, up=B, a=C, saved=act(), ld=50)
    a.update(kw)
    assert lib.muon_swiglu_forward(a["gate"], a["ld"], a["up"], a["ld"], 4, 50, 1, a["a"], a["ld"], a["saved"], None,
                                   None, None) == BAD


@pytest.mark.parametrize("kw", [dict(da=None), dict(g8=None), dict(u8=None), dict(dgate=None), dict(dup=None),
                                dict(dup=B), dict(dgate=A, dup=A), dict(out=act(codes=D, scales=D + 8192))])
def test_swiglu_backward_refuses(lib, kw):
    a = dict(da=A, g8=act(codes=D, scales=D + 4096), u8=act(), dgate=B, dup=C, out=None)
    a.update(kw)
    assert lib.muon_swiglu_backward(a["da"], 50, a["g8"], a["u8"], 4, 50, 1, a["dgate"], 50, a["dup"], 50, a["out"],
                                    None) == BAD


def test_calls_without_a_plan_are_refused(lib):
    assert lib.muon_rmsnorm_backward(None, A, 50, act(), None, 50, C, C + 4096, None, 50, 4, 50, 1, D, 50, None, 0,
                                     None) == BAD
    assert lib.muon_wgrad(None, A, 50, act(), 4, 50, 50, None, 0, None, B, 0, 0, None) == BAD
    assert lib.muon_grad_plan_sync(None, None) == BAD
    assert lib.muon_grad_plan_create(None) == BAD
    assert lib.muon_grad_plan_workspace_size(None) == BAD
    lib.muon_grad_plan_destroy(None)


@pytest.mark.parametrize("kw", [dict(dy=None), dict(x=None), dict(grad=None), dict(grad=A), dict(groups=-1),
                                dict(groups=4097, offsets=C), dict(groups=2), dict(offsets=C), dict(ldy=49),
                                dict(dtype=3), dict(tokens=-1), dict(m=0), dict(n=0), dict(scale=B)])
def test_wgrad_refuses(lib, kw):
    """With a handle that is never read: bad arguments are found first."""
    a = dict(dy=A, ldy=50, x=act(), tokens=4, m=50, n=50, offsets=None, groups=0, scale=None, grad=B, dtype=0)
    a.update(kw)
    fake = ctypes.create_string_buffer(256)
    code = lib.muon_wgrad(ctypes.cast(fake, ctypes.c_void_p), a["dy"], a["ldy"], a["x"], a["tokens"], a["m"], a["n"],
                          a["offsets"], a["groups"], a["scale"], a["grad"], a["dtype"], 0, None)
    assert code == (UNSUP if "dtype" in kw else BAD)


@pytest.mark.parametrize("kw", [dict(saved=None), dict(h=D), dict(dx=None), dict(rstd=None), dict(weight=None),
                                dict(dy=None), dict(dweight=C), dict(dx=C)])
def test_rmsnorm_backward_refuses(lib, kw):
    a = dict(dy=A, saved=act(), h=None, rstd=C, weight=C + 4096, dx=B, dweight=None)
    a.update(kw)
    fake = ctypes.create_string_buffer(256)
    assert lib.muon_rmsnorm_backward(ctypes.cast(fake, ctypes.c_void_p), a["dy"], 50, a["saved"], a["h"], 50, a["rstd"],
                                     a["weight"], None, 50, 4, 50, 0, a["dx"], 50, a["dweight"], 0, None) == BAD


def test_act_layout_matches_the_header():
    import os
    import re
    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "muon.h")).read()
    body = re.search(r"typedef struct \{([^}]*)\}\s*muon_act8\s*;", re.sub(r"/\*.*?\*/", "", src, flags=re.S)).group(1)
    names = [n.strip(" *") for decl in body.split(";") for n in decl.strip().split(" ", 1)[-1].split(",") if decl.strip()]
    assert names == [f for f, _ in mu.MuonAct8._fields_]
    assert ctypes.sizeof(mu.MuonAct8) == 40 and mu.MuonAct8.format.offset == 32


@pytest.mark.parametrize("pitch", [1 << 32, (1 << 32) + 16, 1 << 40])
def test_pitches_of_four_gigabytes_are_refused(lib, pitch):
    assert lib.muon_act_pack(A, 4, 50, pitch // 4, 0, act(), None) == BAD
    assert lib.muon_act_pack(A, 4, 50, 50, 0, act(codes=2 * F, scales=2 * F + (1 << 36), ldq=pitch), None) == BAD


def test_interleaved_halves_do_not_overlap(lib):
    """dgate and dup as the halves of one (rows, 2 cols) tensor pass the overlap check; one column further they
    do not.  (A bad `da` pitch ends the accepted call before it launches.)"""
    def call(dup, ldda):
        return lib.muon_swiglu_backward(A, ldda, act(codes=D, scales=D + 4096), act(), 4, 50, 1, B, 100, dup, 100, None, None)
    assert call(B + 98, 50) == BAD
    if not torch.cuda.is_available():
        assert call(B + 100, 50) == mu.MUON_ERR_CUDA   # passed every check; there is no device to launch on


def test_binding_refuses_tensors_it_cannot_pass():
    x = torch.zeros(4, 50)
    with pytest.raises(ValueError):
        mu.Act8(torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 16, dtype=torch.uint8), 50, "e4m3")   # on the CPU
    with pytest.raises(ValueError):
        mu.Act8.empty(4, 50, "fp4", "cpu")
    with pytest.raises(ValueError):
        mu.rmsnorm_forward(x, torch.ones(50), 1e-6, y=torch.empty(4, 50))
    with pytest.raises(ValueError):
        mu.swiglu_forward(x, x, torch.empty(4, 50))
    with pytest.raises(ValueError):
        mu.rmsnorm_forward(x.double(), torch.ones(50), 1e-6, y=torch.empty(4, 50))
    assert mu.grad_plan_workspace_size() > 0

"""Layer-side operators of the library for torch tensors: activations held in 8 bits
(``Act8``), the RMS norm with the residual's addition, SwiGLU, and, with a ``GradPlan``, the
products of a weight or of experts' weights, the weight gradient that ``MuonPlan.step`` reads,
formed from 8-bit activations, and the norm and clipping of all gradients (``GradList``).

Argument marshalling only, as in the rest of the binding: outputs are the caller's
tensors, work is enqueued on the current stream (or ``stream``), and a call that cannot
run raises.  Two-dimensional CUDA tensors of the current device with unit column stride;
rows may be strided, so column blocks of wider tensors work in place.
"""
from __future__ import annotations

import ctypes

from . import (MUON_ACT_E4M3, MUON_ACT_INT8, MUON_BF16, MUON_F32, MuonAct8, _check, load)

__all__ = ["Act8", "act_pack", "act_unpack", "rmsnorm_forward", "swiglu_forward", "swiglu_backward", "GradPlan",
           "GradList", "grad_plan_workspace_size"]

_FORMATS = {"e4m3": MUON_ACT_E4M3, "int8": MUON_ACT_INT8}
ACT_GROUP = 32
torch = None   # the module and its element types, from the first call on (_torch)
_DTYPES = {}


def _torch():
    """Torch is imported by the first call that takes tensors, as in the rest of the binding."""
    global torch
    import torch as module
    _DTYPES.update({module.float32: MUON_F32, module.bfloat16: MUON_BF16})
    torch = module


def _pad16(n: int) -> int:
    return (n + 15) // 16 * 16


class Act8:
    """An activation of ``rows`` x ``cols`` values in 8 bits (``muon_act8``): ``codes`` and
    ``scales`` are uint8 CUDA tensors whose rows are padded to multiples of 16 bytes; ``fmt``
    is "e4m3" or "int8".  ``Act8.empty`` allocates both."""

    __slots__ = ("codes", "scales", "rows", "cols", "fmt", "device", "ref")

    def __init__(self, codes, scales, cols: int, fmt: str):
        if torch is None:
            _torch()
        if fmt not in _FORMATS:
            raise ValueError("fmt must be 'e4m3' or 'int8', got %r" % (fmt,))
        for t, need, name in ((codes, cols, "codes"), (scales, (cols + ACT_GROUP - 1) // ACT_GROUP, "scales")):
            if t.dtype != torch.uint8 or not t.is_cuda or t.dim() != 2 or t.shape[1] < need or t.stride(1) != 1:
                raise ValueError("%s: need a CUDA uint8 tensor of rows of at least %d bytes, got %s %s"
                                 % (name, need, t.dtype, tuple(t.shape)))
        if codes.shape[0] != scales.shape[0]:
            raise ValueError("codes and scales differ in rows: %d and %d" % (codes.shape[0], scales.shape[0]))
        if codes.get_device() != scales.get_device():
            raise ValueError("codes and scales differ in device: %s and %s" % (codes.device, scales.device))
        self.codes, self.scales, self.rows, self.cols, self.fmt = codes, scales, codes.shape[0], cols, fmt
        self.device = codes.get_device()
        self.ref = MuonAct8(codes.data_ptr(), scales.data_ptr(), self._pitch(codes), self._pitch(scales),
                            _FORMATS[fmt], 0)

    @staticmethod
    def _pitch(t):   # of a single row: one that the library accepts, nothing goes by it
        return t.stride(0) if t.shape[0] > 1 else _pad16(t.shape[1])

    @classmethod
    def empty(cls, rows: int, cols: int, fmt: str = "e4m3", device="cuda") -> "Act8":
        if torch is None:
            _torch()
        groups = (cols + ACT_GROUP - 1) // ACT_GROUP
        return cls(torch.empty((rows, _pad16(cols)), dtype=torch.uint8, device=device),
                   torch.empty((rows, _pad16(groups)), dtype=torch.uint8, device=device), cols, fmt)

    @property
    def nbytes(self) -> int:
        return self.codes.numel() + self.scales.numel()


def _stream(stream, dev):
    """Handle of ``stream``, or of the current stream of device ``dev``."""
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _mat(t, rows, cols, dtype, dev, name):
    """(pointer, row pitch) of one operand, checked."""
    if t is None:
        return None, 0
    if t.dtype is not dtype or t.shape != (rows, cols) or t.get_device() != dev or (cols > 1 and t.stride(1) != 1):
        raise ValueError("%s: need a %s tensor of shape (%d, %d) with unit column stride on the current CUDA device, "
                         "got %s %s strides %s on %s" % (name, dtype, rows, cols, t.dtype, tuple(t.shape),
                                                         tuple(t.stride()), t.device))
    return t.data_ptr(), t.stride(0) if rows > 1 else cols


def _vec(t, n, dev, name, dtype=None):
    if t is None:
        return None
    if dtype is None:
        dtype = torch.float32
    if t.dtype is not dtype or t.shape != (n,) or t.get_device() != dev or (n > 1 and t.stride(0) != 1):
        raise ValueError("%s: need a contiguous %s tensor of %d elements on the current CUDA device, got %s %s on %s"
                         % (name, dtype, n, t.dtype, tuple(t.shape), t.device))
    return t.data_ptr()


def _act(a, rows, cols, dev, name):
    if a is None:
        return None
    if a.rows != rows or a.cols != cols or a.device != dev:
        raise ValueError("%s: need an Act8 of (%d, %d) on the current CUDA device, got (%d, %d) on %s"
                         % (name, rows, cols, a.rows, a.cols, a.codes.device))
    return ctypes.byref(a.ref)


def _shape(t, name):
    """(rows, cols, dtype, dtype code, current device) for the operand that sets a call's shape."""
    if torch is None:
        _torch()
    if t.dim() != 2 or t.dtype not in _DTYPES or not t.is_cuda:
        raise ValueError("%s: need a two-dimensional float32 or bfloat16 CUDA tensor, got %s %s on %s"
                         % (name, t.dtype, tuple(t.shape), t.device))
    rows, cols = t.shape
    return rows, cols, t.dtype, _DTYPES[t.dtype], torch.cuda.current_device()


def act_pack(x, out: Act8, stream=None):
    """``muon_act_pack``: x to 8 bits."""
    rows, cols, dt, code, dev = _shape(x, "x")
    p, ld = _mat(x, rows, cols, dt, dev, "x")
    _check(load().muon_act_pack(p, rows, cols, ld, code, _act(out, rows, cols, dev, "out"), _stream(stream, dev)),
           "muon_act_pack")


def act_unpack(a: Act8, out, stream=None):
    """``muon_act_unpack``: the values of an ``Act8`` into ``out`` (float32 or bfloat16)."""
    rows, cols, dt, code, dev = _shape(out, "out")
    p, ld = _mat(out, rows, cols, dt, dev, "out")
    _check(load().muon_act_unpack(_act(a, rows, cols, dev, "a"), rows, cols, p, ld, code, _stream(stream, dev)),
           "muon_act_unpack")


def rmsnorm_forward(x, weight, eps: float, residual=None, h=None, y=None, saved: Act8 | None = None,
                    saved_weighted: bool = False, rstd=None, stream=None):
    """``muon_rmsnorm_forward``: h = x + residual, y = h / rms(h) * weight; ``saved`` receives the
    norm in 8 bits before the weight (for ``GradPlan``), or y itself with ``saved_weighted``."""
    rows, cols, dt, code, dev = _shape(x, "x")
    px, lx = _mat(x, rows, cols, dt, dev, "x")
    pr, lr = _mat(residual, rows, cols, dt, dev, "residual")
    ph, lh = _mat(h, rows, cols, dt, dev, "h")
    py, ly = _mat(y, rows, cols, dt, dev, "y")
    _check(load().muon_rmsnorm_forward(px, lx, pr, lr, _vec(weight, cols, dev, "weight"), rows, cols, code, eps, ph, lh,
                                       py, ly, _act(saved, rows, cols, dev, "saved"), 1 if saved_weighted else 0,
                                       _vec(rstd, rows, dev, "rstd"), _stream(stream, dev)), "muon_rmsnorm_forward")


def swiglu_forward(gate, up, out=None, saved_gate: Act8 | None = None, saved_up: Act8 | None = None,
                   saved_out: Act8 | None = None, stream=None):
    """``muon_swiglu_forward``: out = silu(gate) * up, with 8-bit copies of any of the three."""
    rows, cols, dt, code, dev = _shape(gate, "gate")
    pg, lg = _mat(gate, rows, cols, dt, dev, "gate")
    pu, lu = _mat(up, rows, cols, dt, dev, "up")
    po, lo = _mat(out, rows, cols, dt, dev, "out")
    _check(load().muon_swiglu_forward(pg, lg, pu, lu, rows, cols, code, po, lo,
                                      _act(saved_gate, rows, cols, dev, "saved_gate"),
                                      _act(saved_up, rows, cols, dev, "saved_up"),
                                      _act(saved_out, rows, cols, dev, "saved_out"), _stream(stream, dev)),
           "muon_swiglu_forward")


def swiglu_backward(dout, saved_gate: Act8, saved_up: Act8, dgate, dup, saved_out: Act8 | None = None, stream=None):
    """``muon_swiglu_backward``: dgate and dup from dout and the 8-bit gate and up; ``saved_out``
    receives silu(gate) * up again in 8 bits, the operand of the down projection's gradient."""
    rows, cols, dt, code, dev = _shape(dout, "dout")
    pd, ldd = _mat(dout, rows, cols, dt, dev, "dout")
    pg, lg = _mat(dgate, rows, cols, dt, dev, "dgate")
    pu, lu = _mat(dup, rows, cols, dt, dev, "dup")
    _check(load().muon_swiglu_backward(pd, ldd, _act(saved_gate, rows, cols, dev, "saved_gate"),
                                       _act(saved_up, rows, cols, dev, "saved_up"), rows, cols, code, pg, lg, pu, lu,
                                       _act(saved_out, rows, cols, dev, "saved_out"), _stream(stream, dev)),
           "muon_swiglu_backward")


def grad_plan_workspace_size(aligned_bytes: int | None = None) -> int:
    """Device bytes that a ``GradPlan`` of these ``aligned_bytes`` allocates (``muon_grad_plan_workspace_size``; no GPU
    needed)."""
    n = ctypes.c_int64()
    if aligned_bytes is None:
        _check(load().muon_grad_plan_workspace_size(ctypes.byref(n)), "muon_grad_plan_workspace_size")
    else:
        _check(load().muon_grad_plan_workspace_size_ex(aligned_bytes, ctypes.byref(n)), "muon_grad_plan_workspace_size_ex")
    return n.value


class GradList:
    """Gradients of any shapes, fp32 or bf16, dense, as ``GradPlan.grad_norm`` and ``GradPlan.grad_clip`` take them:
    their pointers, counts and types, gathered once (a list that is built anew for every call costs the host about
    a microsecond per tensor).  It keeps the tensors alive."""

    __slots__ = ("tensors", "device", "n", "pointers", "counts", "dtypes")

    def __init__(self, tensors):
        if torch is None:
            _torch()
        self.tensors = list(tensors)
        self.device = self.tensors[0].get_device() if self.tensors else torch.cuda.current_device()
        for i, t in enumerate(self.tensors):
            if t.dtype not in _DTYPES or not t.is_cuda or not t.is_contiguous() or t.get_device() != self.device:
                raise ValueError("gradient %d: need a contiguous float32 or bfloat16 CUDA tensor on %s, got %s %s on %s"
                                 % (i, self.device, t.dtype, tuple(t.shape), t.device))
        self.n = len(self.tensors)
        self.pointers = (ctypes.c_void_p * self.n)(*[t.data_ptr() for t in self.tensors])
        self.counts = (ctypes.c_int64 * self.n)(*[t.numel() for t in self.tensors])
        self.dtypes = (ctypes.c_int32 * self.n)(*[_DTYPES[t.dtype] for t in self.tensors])


def _grads(grads, dev, name):
    grads = grads if isinstance(grads, GradList) else GradList(grads)
    if grads.device != dev:
        raise ValueError("%s: need gradients on the current CUDA device, got them on %s" % (name, grads.device))
    return grads


class GradPlan:
    """Workspace and status word of the reductions and products on the current device
    (``muon_grad_plan_create``); one serves calls of any shapes, one after another.  ``aligned_bytes``: the part of the
    workspace for copies of unaligned rows alone, which only ``product`` and ``dgrad`` make (0: the smallest plan, on
    which large products of such rows are slower)."""

    def __init__(self, aligned_bytes: int | None = None):
        if torch is None:
            _torch()
        self.lib = load()
        h = ctypes.c_void_p()
        if aligned_bytes is None:
            _check(self.lib.muon_grad_plan_create(ctypes.byref(h)), "muon_grad_plan_create")
        else:
            _check(self.lib.muon_grad_plan_create_ex(ctypes.byref(h), aligned_bytes), "muon_grad_plan_create_ex")
        self.handle = h

    def close(self):
        if getattr(self, "handle", None):
            self.lib.muon_grad_plan_destroy(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def sync(self, stream=None):
        """``muon_grad_plan_sync``: wait for the stream and raise what the device reported."""
        _check(self.lib.muon_grad_plan_sync(self.handle, _stream(stream, torch.cuda.current_device())),
               "muon_grad_plan_sync")

    def rmsnorm_backward(self, dy, weight, rstd, dx=None, dweight=None, saved: Act8 | None = None, h=None, dres=None,
                         accumulate: bool = False, stream=None):
        """``muon_rmsnorm_backward`` from ``saved`` (the unweighted norm in 8 bits) or ``h``."""
        rows, cols, dt, code, dev = _shape(dy, "dy")
        py, ly = _mat(dy, rows, cols, dt, dev, "dy")
        ph, lh = _mat(h, rows, cols, dt, dev, "h")
        pr, lr = _mat(dres, rows, cols, dt, dev, "dres")
        px, lx = _mat(dx, rows, cols, dt, dev, "dx")
        _check(self.lib.muon_rmsnorm_backward(self.handle, py, ly, _act(saved, rows, cols, dev, "saved"), ph, lh,
                                              _vec(rstd, rows, dev, "rstd"), _vec(weight, cols, dev, "weight"), pr, lr, rows,
                                              cols, code, px, lx, _vec(dweight, cols, dev, "dweight"),
                                              1 if accumulate else 0, _stream(stream, dev)),
               "muon_rmsnorm_backward")

    def wgrad(self, dy, x: Act8, grad, offsets=None, col_scale=None, accumulate: bool = False, stream=None):
        """``muon_wgrad``: grad (m, n) (+)= dy^T x * col_scale, dy (tokens, m) bfloat16, x (tokens, n)
        in 8 bits; with ``offsets`` (groups + 1 int32, on the device) grad is (groups, m, n), one
        weight per range of tokens."""
        dev = torch.cuda.current_device()
        if dy.dim() != 2 or grad.dtype not in _DTYPES:
            raise ValueError("wgrad: need a two-dimensional dy and a float32 or bfloat16 grad, got %s and %s"
                             % (tuple(dy.shape), grad.dtype))
        (tokens, m), n = dy.shape, x.cols
        groups = 0 if offsets is None else offsets.numel() - 1
        shape = (m, n) if offsets is None else (groups, m, n)
        if grad.shape != shape or not grad.is_contiguous() or grad.get_device() != dev \
                or groups < (offsets is not None):
            raise ValueError("grad: need a contiguous tensor of shape %s on the current CUDA device, got %s on %s"
                             % (shape, tuple(grad.shape), grad.device))
        py, ly = _mat(dy, tokens, m, torch.bfloat16, dev, "dy")
        _check(self.lib.muon_wgrad(self.handle, py, ly, _act(x, tokens, n, dev, "x"), tokens, m, n,
                                   _vec(offsets, groups + 1, dev, "offsets", torch.int32), groups,
                                   _vec(col_scale, n, dev, "col_scale"), grad.data_ptr(), _DTYPES[grad.dtype],
                                   1 if accumulate else 0, _stream(stream, dev)), "muon_wgrad")

    def _product(self, name, x, weight, out, offsets, dgrad, stream):
        dev = torch.cuda.current_device()
        groups = 0 if offsets is None else offsets.numel() - 1
        if x.dim() != 2 or weight.dim() != (2 if offsets is None else 3) or weight.dtype is not torch.bfloat16 \
                or not weight.is_contiguous() or weight.get_device() != dev or groups < (offsets is not None) \
                or (groups and weight.shape[0] != groups):
            raise ValueError("%s: need a two-dimensional input and a contiguous bfloat16 weight %s on the current CUDA "
                             "device, got %s and %s %s on %s" % (name, "(m, n)" if offsets is None else
                                                                 "(%d, m, n)" % groups, tuple(x.shape), weight.dtype,
                                                                 tuple(weight.shape), weight.device))
        tokens, (m, n) = x.shape[0], weight.shape[-2:]
        px, lx = _mat(x, tokens, m if dgrad else n, torch.bfloat16, dev, "dy" if dgrad else "x")
        po, lo = _mat(out, tokens, n if dgrad else m, torch.bfloat16, dev, "dx" if dgrad else "out")
        _check(getattr(self.lib, name)(self.handle, px, lx, weight.data_ptr(), tokens, m, n,
                                       _vec(offsets, groups + 1, dev, "offsets", torch.int32), groups, po, lo,
                                       _stream(stream, dev)), name)

    def product(self, x, weight, out, offsets=None, stream=None):
        """``muon_product``: out (tokens, m) = x (tokens, n) W^T, bfloat16, weight (m, n); with ``offsets`` (groups + 1
        int32, on the device) weight is (groups, m, n), one per range of tokens, and rows outside them are left."""
        self._product("muon_product", x, weight, out, offsets, False, stream)

    def dgrad(self, dy, weight, dx, offsets=None, stream=None):
        """``muon_dgrad``: dx (tokens, n) = dy (tokens, m) W, the gradient of ``product``'s input."""
        self._product("muon_dgrad", dy, weight, dx, offsets, True, stream)

    def grad_norm(self, grads, norm, stream=None):
        """``muon_grad_norm``: norm (one float32, on the device) of all gradients of ``grads`` (a ``GradList`` or
        tensors) together."""
        dev = torch.cuda.current_device()
        g = _grads(grads, dev, "grad_norm")
        _check(self.lib.muon_grad_norm(self.handle, g.pointers, g.counts, g.dtypes, g.n, _vec(norm, 1, dev, "norm"),
                                       _stream(stream, dev)), "muon_grad_norm")

    def grad_clip(self, grads, norm, max_norm: float, out=None, stream=None):
        """``muon_grad_clip``: the gradients times max_norm / norm where norm > max_norm, in place or into the
        tensors of ``out``, which may be of the other type."""
        dev = torch.cuda.current_device()
        g = _grads(grads, dev, "grad_clip")
        o = None if out is None else _grads(out, dev, "grad_clip")
        if o is not None and bytes(o.counts) != bytes(g.counts):
            raise ValueError("out: need tensors of the gradients' sizes")
        _check(self.lib.muon_grad_clip(self.handle, g.pointers, g.counts, g.dtypes, g.n, _vec(norm, 1, dev, "norm"),
                                       max_norm, None if o is None else o.pointers, None if o is None else o.dtypes,
                                       _stream(stream, dev)), "muon_grad_clip")

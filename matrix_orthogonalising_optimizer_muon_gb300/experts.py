"""Tokens in their experts' order and back, for torch tensors: ``expert_order``,
``expert_dispatch``, ``expert_combine`` and ``expert_combine_backward``.  ``offsets`` is what
``GradPlan.product``, ``GradPlan.dgrad`` and ``GradPlan.wgrad`` take; ``slots`` (tokens, choices)
says in which row of the experts' order each choice of a token stands.

Argument marshalling only, as in ``activations``.
"""
from __future__ import annotations

from . import _check, activations, load
from .activations import _mat, _shape, _stream, _vec

__all__ = ["expert_order", "expert_dispatch", "expert_combine", "expert_combine_backward"]


def _table(t, shape, dtype, dev, name):
    """Pointer of a dense (tokens, choices) table, checked; None for None."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        raise ValueError("%s: need a contiguous %s tensor of shape %s on the current CUDA device, got %s %s on %s"
                         % (name, dtype, tuple(shape), t.dtype, tuple(t.shape), t.device))
    return t.data_ptr()


def _choices(slots, dev, name="slots"):
    """(pointer, tokens, choices) of the table that sets a call's tokens and choices."""
    if slots.dim() != 2:
        raise ValueError("%s: need a (tokens, choices) tensor, got %s" % (name, tuple(slots.shape)))
    return _table(slots, slots.shape, activations.torch.int32, dev, name), slots.shape[0], slots.shape[1]


def expert_order(ids, offsets, slots, stream=None):
    """``muon_expert_order``: ids (tokens, choices) int32, the experts of each token (a value outside them is
    no choice), to offsets (experts + 1) and slots (tokens, choices), int32."""
    if activations.torch is None:
        activations._torch()
    i32, dev = activations.torch.int32, activations.torch.cuda.current_device()
    p, tokens, choices = _choices(ids, dev, "ids")
    if offsets.dim() != 1 or offsets.numel() < 2:
        raise ValueError("offsets: need experts + 1 values, got %s" % (tuple(offsets.shape),))
    _check(load().muon_expert_order(p, tokens, choices, offsets.numel() - 1,
                                    _vec(offsets, offsets.numel(), dev, "offsets", i32),
                                    _table(slots, ids.shape, i32, dev, "slots"), _stream(stream, dev)),
           "muon_expert_order")


def expert_dispatch(x, slots, out, stream=None):
    """``muon_expert_dispatch``: out[slots[t, j]] = x[t]; other rows of out are left as they were."""
    tokens, cols, dt, code, dev = _shape(x, "x")
    ps, _, choices = _choices(slots, dev)
    if slots.shape[0] != tokens:
        raise ValueError("slots: need %d tokens, got %s" % (tokens, tuple(slots.shape)))
    rows = out.shape[0]
    px, lx = _mat(x, tokens, cols, dt, dev, "x")
    po, lo = _mat(out, rows, cols, dt, dev, "out")
    _check(load().muon_expert_dispatch(px, lx, ps, tokens, choices, rows, cols, code, po, lo, _stream(stream, dev)),
           "muon_expert_dispatch")


def expert_combine(rows, slots, out, weights=None, stream=None):
    """``muon_expert_combine``: out[t] = sum over j of weights[t, j] * rows[slots[t, j]] (weights None: ones, the
    gradient of ``expert_dispatch``)."""
    tokens, cols, dt, code, dev = _shape(out, "out")
    ps, _, choices = _choices(slots, dev)
    if slots.shape[0] != tokens:
        raise ValueError("slots: need %d tokens, got %s" % (tokens, tuple(slots.shape)))
    n = rows.shape[0]
    po, lo = _mat(out, tokens, cols, dt, dev, "out")
    pr, lr = _mat(rows, n, cols, dt, dev, "rows")
    _check(load().muon_expert_combine(pr, lr, ps, _table(weights, slots.shape, activations.torch.float32, dev, "weights"),
                                      tokens, choices, n, cols, code, po, lo, _stream(stream, dev)),
           "muon_expert_combine")


def expert_combine_backward(dout, slots, weights, rows=None, drows=None, dweights=None, stream=None):
    """``muon_expert_combine_backward``: drows[slots[t, j]] = weights[t, j] * dout[t], other rows left as they were,
    and dweights[t, j] = dout[t] . rows[slots[t, j]] (either may be None; rows is read for dweights alone, which
    needs it)."""
    tokens, cols, dt, code, dev = _shape(dout, "dout")
    ps, _, choices = _choices(slots, dev)
    if slots.shape[0] != tokens:
        raise ValueError("slots: need %d tokens, got %s" % (tokens, tuple(slots.shape)))
    given = rows if rows is not None else drows
    # where neither says how many rows there are, slots may name any: dweights without rows is refused, as beside drows
    n = given.shape[0] if given is not None else slots.numel()
    f32 = activations.torch.float32
    pd, ld = _mat(dout, tokens, cols, dt, dev, "dout")
    pr, lr = _mat(rows, n, cols, dt, dev, "rows")
    pg, lg = _mat(drows, n, cols, dt, dev, "drows")
    _check(load().muon_expert_combine_backward(pd, ld, ps, _table(weights, slots.shape, f32, dev, "weights"), pr, lr,
                                               tokens, choices, n, cols, code, pg, lg,
                                               _table(dweights, slots.shape, f32, dev, "dweights"),
                                               _stream(stream, dev)), "muon_expert_combine_backward")

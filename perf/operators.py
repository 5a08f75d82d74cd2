"""Cases of the training-side operators around a weight that Muon updates: the
root-mean-square norm with the residual's addition, the gated activation, activations
held in 8 bits between the forward and the backward pass, and the weight gradient
formed from them.

``run`` computes an operator in its plain form (elementary torch operations in 32
bits, rounded once at the end), or, where ``own`` is true, through the framework's
entry points.  ``exact`` gives the same outputs from the definitions in 64 bits.

An activation in 8 bits (``Act8``): one code per value and one power-of-two scale per
32 neighbouring values of a row, stored as its biased exponent (value 2^(byte - 127),
255: a group that held an infinity or a NaN).  Codes are e4m3 numbers ("e4m3") or
whole numbers -127..127 ("int8").  The scale is the smallest 2^e with which the group's
largest magnitude fits the codes.  Rows of codes and of scales are padded to multiples
of 16 bytes.
"""
import math

import torch

own = False

GROUP = 32
EPS = 1e-6
LOWEST = -110                              # smallest scale exponent
HIGHEST = {"e4m3": 119, "int8": 121}       # largest scale exponent
LARGEST = {"e4m3": 448.0, "int8": 127.0}   # largest code

_kept = {}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one token's norm on its way into an 8-bit product: latency alone
        {"name": "norm_fwd_one_token", "op": "norm_fwd", "rows": 1, "cols": 3584, "dtype": "bf16", "fmt": "e4m3",
         "residual": True, "weighted": True},
        # a training micro-batch of 16k tokens at hidden 3584
        {"name": "norm_fwd_16k", "op": "norm_fwd", "rows": 16384, "cols": 3584, "dtype": "bf16", "fmt": "e4m3",
         "residual": True, "weighted": False},
        # its backward pass from the 8-bit copy, with the gradient that comes down the residual path
        {"name": "norm_bwd_16k", "op": "norm_bwd", "rows": 16384, "cols": 3584, "dtype": "bf16", "fmt": "int8",
         "residual": True, "from8": True},
        # fp32 training of a small model with an odd width, from the full activation
        {"name": "norm_bwd_odd_f32", "op": "norm_bwd", "rows": 777, "cols": 1001, "dtype": "f32", "fmt": "e4m3",
         "residual": True, "from8": False},
        # the gated activation of an FFN of 18944, gate and up the halves of one product's output
        {"name": "glu_fwd_8k", "op": "glu_fwd", "rows": 8192, "cols": 18944, "dtype": "bf16", "fmt": "e4m3"},
        # its backward pass, which also rebuilds the 8-bit input of the down projection's gradient
        {"name": "glu_bwd_8k", "op": "glu_bwd", "rows": 8192, "cols": 18944, "dtype": "bf16", "fmt": "e4m3"},
        # a few tokens' activation written to 8 bits and read back, odd width
        {"name": "pack_small_odd", "op": "pack", "rows": 65, "cols": 1001, "dtype": "f32", "fmt": "int8"},
        # a layer's activations at 32k tokens, a column block of a wider tensor
        {"name": "pack_32k", "op": "pack", "rows": 32768, "cols": 2048, "dtype": "bf16", "fmt": "int8"},
        # a small weight with odd sides and a short batch, added to the gradient of earlier micro-batches
        {"name": "wgrad_small_odd", "op": "wgrad", "rows": 257, "m": 515, "n": 1001, "groups": 0, "fmt": "int8",
         "dtype": "f32", "accumulate": True, "scaled": False},
        # an attention projection at hidden 3584, bf16 gradient, the norm's weight folded in
        {"name": "wgrad_8k_square", "op": "wgrad", "rows": 8192, "m": 3584, "n": 3584, "groups": 0, "fmt": "int8",
         "dtype": "bf16", "accumulate": False, "scaled": True},
        # an FFN projection over 16k tokens, fp32 gradient
        {"name": "wgrad_16k_ffn", "op": "wgrad", "rows": 16384, "m": 18944, "n": 3584, "groups": 0, "fmt": "e4m3",
         "dtype": "f32", "accumulate": False, "scaled": True},
        # 32 experts' weights from tokens sorted by expert: ragged lengths, some experts without a token
        {"name": "wgrad_experts", "op": "wgrad", "rows": 16384, "m": 1024, "n": 2048, "groups": 32, "fmt": "e4m3",
         "dtype": "bf16", "accumulate": False, "scaled": False},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over the logarithm; half of them odd as drawn, half rounded to 64."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5 and v >= 64:
        v = (v + 32) // 64 * 64
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "glu_fwd", "glu_bwd", "pack", "wgrad", "wgrad"])
    fmt = rng.choice(["e4m3", "int8"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "wgrad":
        groups = rng.choice([0, 0, _spread(rng, 2, 64)])
        m, n = _spread(rng, 128, 8192 if not groups else 2048), _spread(rng, 128, 8192 if not groups else 2048)
        return {"op": op, "rows": _spread(rng, 1, 16384), "m": m, "n": n, "groups": groups, "fmt": fmt,
                "dtype": rng.choice(["bf16", "f32"]), "accumulate": rng.random() < 0.4, "scaled": rng.random() < 0.5}
    cols = _spread(rng, 32, 8192 if op.startswith("norm") else 18944)
    case = {"op": op, "rows": _spread(rng, 1, max(1, min(32768, 60_000_000 // cols))), "cols": cols, "dtype": dtype,
            "fmt": fmt}
    if op == "norm_fwd":
        # whole-number codes are read back through another operator; here the outputs are the 8-bit floats
        case.update(fmt="e4m3", residual=rng.random() < 0.7, weighted=rng.random() < 0.5)
    elif op == "norm_bwd":
        case.update(residual=rng.random() < 0.7, from8=rng.random() < 0.7)
    elif op in ("glu_fwd", "glu_bwd"):
        case.update(fmt="e4m3")
    return case


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    t = case["rows"]
    q = 1 + 1 / GROUP   # one code and its share of the scale
    if case["op"] == "wgrad":
        m, n, g = case["m"], case["n"], max(1, case["groups"])
        out = g * m * n * e * (2 if case["accumulate"] else 1)
        return {"bytes": t * m * 2 + t * n * q + out + (4 * n if case["scaled"] else 0), "flops": 2.0 * t * m * n}
    c = case["cols"]
    if case["op"] == "norm_fwd":
        per = e * (1 + 1 + (2 if case["residual"] else 0)) + q
        return {"bytes": t * c * per + 4 * (c + t), "flops": 8.0 * t * c}
    if case["op"] == "norm_bwd":
        per = e * (1 + 1 + (1 if case["residual"] else 0)) + (q if case["from8"] else e)
        return {"bytes": t * c * per + 4 * (2 * c + t), "flops": 10.0 * t * c}
    if case["op"] == "glu_fwd":
        return {"bytes": t * c * (3 * e + 2 * q), "flops": 10.0 * t * c}
    if case["op"] == "glu_bwd":
        return {"bytes": t * c * (3 * e + 3 * q), "flops": 16.0 * t * c}
    return {"bytes": t * c * (2 * e + 2 * q), "flops": 4.0 * t * c}


# ---------------------------------------------------------------- inputs
def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 64 + salt)
    return g


def _dt(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _there(rows, seed):
    """0 for the tokens that pad the batch (about one in a hundred), else 1: they have no activation and no gradient."""
    if rows < 16:
        return torch.ones((rows, 1), device="cuda")
    return (torch.rand((rows, 1), generator=_gen(seed, 63), device="cuda") >= 0.01).float()


def _activation(rows, cols, seed, salt, dtype):
    """Activations: a few channels far larger than the rest, tokens of unequal size, padding tokens of zeros."""
    g = _gen(seed, salt)
    x = torch.randn((rows, cols), generator=g, device="cuda")
    channel = torch.exp(0.5 * torch.randn((1, cols), generator=g, device="cuda"))
    channel = torch.where(torch.rand((1, cols), generator=g, device="cuda") < 0.002, 20.0 * channel, channel)
    token = torch.exp(0.3 * torch.randn((rows, 1), generator=g, device="cuda"))
    return (x * channel * token * _there(rows, seed)).to(dtype)


def _gradient(rows, cols, seed, salt, dtype, scale=1e-2):
    g = _gen(seed, salt)
    x = torch.randn((rows, cols), generator=g, device="cuda")
    token = torch.exp(0.5 * torch.randn((rows, 1), generator=g, device="cuda"))
    return (x * token * scale * _there(rows, seed)).to(dtype)


def _pad16(n):
    return (n + 15) // 16 * 16


def _held(values, fmt):
    """The codes and scales that a forward pass left: values [rows, cols] in 32 bits -> two byte tensors, padded rows."""
    rows, cols = values.shape
    codes, byte = _codes(values, fmt)
    q = torch.zeros((rows, _pad16(cols)), dtype=torch.uint8, device=values.device)
    s = torch.zeros((rows, _pad16(byte.shape[1])), dtype=torch.uint8, device=values.device)
    q[:, :cols] = codes
    s[:, :byte.shape[1]] = byte
    return q, s


def _empty_held(rows, cols):
    return (torch.zeros((rows, _pad16(cols)), dtype=torch.uint8, device="cuda"),
            torch.zeros((rows, _pad16((cols + GROUP - 1) // GROUP)), dtype=torch.uint8, device="cuda"))


def _lengths(rows, groups, seed):
    """Tokens of each expert: uneven shares that sum to `rows`, about one expert in eight without any."""
    import random
    r = random.Random(seed)
    share = [0.0 if r.random() < 0.125 else r.expovariate(1.0) + 0.05 for _ in range(groups)]
    if not any(share):
        share[0] = 1.0
    edges, acc, total = [0], 0.0, sum(share)
    for x in share:
        acc += x
        edges.append(int(round(rows * acc / total)))
    edges[-1] = rows
    return edges


def prepare(case, seed):
    op, t, dt = case["op"], case["rows"], _dt(case)
    s = {"case": case}
    if own:
        import matrix_orthogonalising_optimizer_muon_gb300 as muon
        if "plan" not in _kept:
            _kept["plan"] = muon.GradPlan()      # one plan serves every call of a program
        s["muon"], s["plan"] = muon, _kept["plan"]
    if op == "wgrad":
        m, n, groups = case["m"], case["n"], case["groups"]
        s["dy"] = _gradient(t, m, seed, 1, torch.bfloat16)
        s["x8"] = _held(_activation(t, n, seed, 2, torch.float32), case["fmt"])
        shape = (groups, m, n) if groups else (m, n)
        if case["accumulate"]:
            s["grad"] = (torch.randn(shape, generator=_gen(seed, 3), device="cuda") * 1e-2).to(dt)
        else:
            s["grad"] = torch.empty(shape, dtype=dt, device="cuda")
        s["scale"] = 1 + 0.2 * torch.randn((n,), generator=_gen(seed, 4), device="cuda") if case["scaled"] else None
        s["offsets"] = None
        if groups:
            edges = _lengths(t, groups, seed)
            s["offsets"] = torch.tensor(edges, dtype=torch.int32, device="cuda")
            s["longest"] = max(b - a for a, b in zip(edges, edges[1:]))
        return s
    c = case["cols"]
    if op == "norm_fwd":
        s["x"] = _activation(t, c, seed, 1, dt)
        s["residual"] = _activation(t, c, seed, 2, dt) if case["residual"] else None
        s["weight"] = 1 + 0.2 * torch.randn((c,), generator=_gen(seed, 3), device="cuda")
        s["h"] = torch.empty_like(s["x"]) if case["residual"] else None
        s["y"], s["rstd"] = torch.empty_like(s["x"]), torch.empty((t,), device="cuda")
        s["saved"] = _empty_held(t, c)
    elif op == "norm_bwd":
        h = _activation(t, c, seed, 1, dt)
        s["weight"] = 1 + 0.2 * torch.randn((c,), generator=_gen(seed, 3), device="cuda")
        s["rstd"] = torch.rsqrt(h.float().square().mean(1) + EPS)
        s["saved"] = _held(h.float() * s["rstd"][:, None], case["fmt"]) if case["from8"] else None
        s["h"] = None if case["from8"] else h
        s["dy"] = _gradient(t, c, seed, 4, dt)
        s["dres"] = _gradient(t, c, seed, 5, dt) if case["residual"] else None
        s["dx"], s["dweight"] = torch.empty_like(s["dy"]), torch.empty((c,), device="cuda")
    elif op == "glu_fwd":
        s["gu"] = _activation(t, 2 * c, seed, 1, dt)
        s["a"] = torch.empty((t, c), dtype=dt, device="cuda")
        s["g8"], s["u8"] = _empty_held(t, c), _empty_held(t, c)
    elif op == "glu_bwd":
        s["g8"] = _held(_activation(t, c, seed, 1, torch.float32), case["fmt"])
        s["u8"] = _held(_activation(t, c, seed, 2, torch.float32), case["fmt"])
        s["da"] = _gradient(t, c, seed, 4, dt)
        s["dgu"] = torch.empty((t, 2 * c), dtype=dt, device="cuda")
        s["a8"] = _empty_held(t, c)
    else:
        s["wide"] = _activation(t, c + 64, seed, 1, dt)   # the packed columns lie inside a wider tensor
        s["saved"], s["back"] = _empty_held(t, c), torch.empty((t, c), dtype=dt, device="cuda")
    return s


# ---------------------------------------------------------------- plain forms
def _codes(v, fmt):
    """Codes [rows, cols] as bytes and scale bytes [rows, groups] of values in 32 bits."""
    rows, cols = v.shape
    n = (cols + GROUP - 1) // GROUP
    if n * GROUP != cols:
        v = torch.nn.functional.pad(v, (0, n * GROUP - cols))
    v = v.reshape(rows, n, GROUP)
    amax = v.abs().amax(2)
    bad = ~torch.isfinite(amax)
    f, k = torch.frexp(torch.where(bad, torch.ones_like(amax), amax))     # amax = f 2^k, 1/2 <= f < 1
    e = k - 9 + (f > 0.875) if fmt == "e4m3" else k - 7 + (f > 127 / 128)
    e = torch.where(amax == 0, torch.full_like(e, LOWEST), e).clamp(LOWEST, HIGHEST[fmt])
    w = v * torch.exp2(-e.float())[:, :, None]
    w = torch.where(bad[:, :, None], torch.zeros_like(w), w).clamp(-LARGEST[fmt], LARGEST[fmt])
    if fmt == "e4m3":
        q = w.to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        q = torch.round(w).to(torch.int8).view(torch.uint8)
    byte = torch.where(bad, torch.full_like(e, 255), e + 127).to(torch.uint8)
    return q.reshape(rows, n * GROUP)[:, :cols], byte


def _values(held, cols, fmt):
    """What codes and scales stand for, in 32 bits."""
    q, s = held[0][:, :cols], held[1][:, :(cols + GROUP - 1) // GROUP]
    q = q.contiguous().view(torch.float8_e4m3fn if fmt == "e4m3" else torch.int8).float()
    scale = torch.where(s == 255, torch.full((), float("nan"), device=s.device), torch.exp2(s.float() - 127))
    return q * scale.repeat_interleave(GROUP, 1)[:, :cols]


def _store(held, v, fmt):
    codes, byte = _codes(v, fmt)
    held[0][:, :codes.shape[1]] = codes
    held[1][:, :byte.shape[1]] = byte


def _read(held, cols):
    """e4m3 codes and their scales as the numbers they are."""
    return {"codes": held[0].view(torch.float8_e4m3fn)[:, :cols],
            "scales": held[1].view(torch.float8_e8m0fnu)[:, :(cols + GROUP - 1) // GROUP]}


def _plain(s):
    case = s["case"]
    op, dt = case["op"], _dt(case)
    if op == "wgrad":
        n = case["n"]
        x, dy = _values(s["x8"], n, case["fmt"]), s["dy"].float()
        if case["groups"]:
            start, end = s["offsets"][:-1].long()[:, None], s["offsets"][1:].long()[:, None]
            at = start + torch.arange(s["longest"], device="cuda")[None]          # token of (expert, place)
            there = (at < end)[:, :, None]
            at = at.clamp(max=case["rows"] - 1)
            zero = torch.zeros((), device="cuda")
            g = torch.bmm(torch.where(there, dy[at], zero).transpose(1, 2), torch.where(there, x[at], zero))
        else:
            g = dy.t() @ x
        if s["scale"] is not None:
            g = g * s["scale"]
        if case["accumulate"]:
            g = g + s["grad"].float()
        s["grad"].copy_(g)
        return {"grad": s["grad"]}
    c = case["cols"]
    if op == "norm_fwd":
        h = s["x"].float()
        if case["residual"]:
            h = h + s["residual"].float()
            s["h"].copy_(h)
        rstd = torch.rsqrt(h.square().mean(1) + EPS)
        s["rstd"].copy_(rstd)
        xhat = h * rstd[:, None]
        y = xhat * s["weight"]
        s["y"].copy_(y)
        _store(s["saved"], y if case["weighted"] else xhat, case["fmt"])
        return {"h": s["h"], "y": s["y"], "rstd": s["rstd"], "saved": _read(s["saved"], c)}
    if op == "norm_bwd":
        xhat = _values(s["saved"], c, case["fmt"]) if case["from8"] else s["h"].float() * s["rstd"][:, None]
        dy = s["dy"].float()
        w = dy * s["weight"]
        dx = (w - xhat * (w * xhat).mean(1, keepdim=True)) * s["rstd"][:, None]
        if case["residual"]:
            dx = dx + s["dres"].float()
        s["dx"].copy_(dx)
        s["dweight"].copy_((dy * xhat).sum(0))
        return {"dx": s["dx"], "dweight": s["dweight"]}
    if op == "glu_fwd":
        gate, up = s["gu"][:, :c].float(), s["gu"][:, c:].float()
        s["a"].copy_(gate * torch.sigmoid(gate) * up)
        _store(s["g8"], gate, case["fmt"])
        _store(s["u8"], up, case["fmt"])
        return {"a": s["a"], "gate": _read(s["g8"], c), "up": _read(s["u8"], c)}
    if op == "glu_bwd":
        gate, up = _values(s["g8"], c, case["fmt"]), _values(s["u8"], c, case["fmt"])
        da = s["da"].float()
        sig = torch.sigmoid(gate)
        silu = gate * sig
        s["dgu"][:, :c] = (da * up * (sig + silu * (1 - sig))).to(dt)
        s["dgu"][:, c:] = (da * silu).to(dt)
        _store(s["a8"], silu * up, case["fmt"])
        return {"dgu": s["dgu"], "a": _read(s["a8"], c)}
    _store(s["saved"], s["wide"][:, 32:32 + c].float(), case["fmt"])
    s["back"].copy_(_values(s["saved"], c, case["fmt"]))
    return {"back": s["back"]}


# ---------------------------------------------------------------- the framework's calls
def _own(s):
    case, muon, plan = s["case"], s["muon"], s["plan"]
    op = case["op"]
    if op == "wgrad":
        plan.wgrad(s["dy"], muon.Act8(*s["x8"], case["n"], case["fmt"]), s["grad"], offsets=s["offsets"],
                   col_scale=s["scale"], accumulate=case["accumulate"])
        return {"grad": s["grad"]}
    c, fmt = case["cols"], case["fmt"]
    if op == "norm_fwd":
        muon.rmsnorm_forward(s["x"], s["weight"], EPS, residual=s["residual"], h=s["h"], y=s["y"],
                             saved=muon.Act8(*s["saved"], c, fmt), saved_weighted=case["weighted"], rstd=s["rstd"])
        return {"h": s["h"], "y": s["y"], "rstd": s["rstd"], "saved": _read(s["saved"], c)}
    if op == "norm_bwd":
        plan.rmsnorm_backward(s["dy"], s["weight"], s["rstd"], s["dx"], dweight=s["dweight"],
                              saved=muon.Act8(*s["saved"], c, fmt) if case["from8"] else None, h=s["h"],
                              dres=s["dres"])
        return {"dx": s["dx"], "dweight": s["dweight"]}
    if op == "glu_fwd":
        muon.swiglu_forward(s["gu"][:, :c], s["gu"][:, c:], s["a"], saved_gate=muon.Act8(*s["g8"], c, fmt),
                            saved_up=muon.Act8(*s["u8"], c, fmt))
        return {"a": s["a"], "gate": _read(s["g8"], c), "up": _read(s["u8"], c)}
    if op == "glu_bwd":
        muon.swiglu_backward(s["da"], muon.Act8(*s["g8"], c, fmt), muon.Act8(*s["u8"], c, fmt), s["dgu"][:, :c],
                             s["dgu"][:, c:], saved_out=muon.Act8(*s["a8"], c, fmt))
        return {"dgu": s["dgu"], "a": _read(s["a8"], c)}
    held = muon.Act8(*s["saved"], c, fmt)
    muon.act_pack(s["wide"][:, 32:32 + c], held)
    muon.act_unpack(held, s["back"])
    return {"back": s["back"]}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- definitions in 64 bits
def _two(e):
    """2^e in 64 bits, exactly, for whole e of the normal range."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _round64(x, fmt):
    """x (64 bits, any shape whose last axis is one row) -> (codes, scales) as numbers in 64 bits."""
    rows, cols = x.shape
    n = -(-cols // GROUP)
    z = x.new_zeros((rows, n * GROUP))
    z[:, :cols] = x
    z = z.view(rows, n, GROUP)
    big = z.abs().max(dim=2).values
    # smallest e with big <= LARGEST 2^e
    e = torch.ceil(torch.log2(big.clamp(min=1e-300) / LARGEST[fmt]))
    e = torch.where(big > LARGEST[fmt] * _two(e), e + 1, e)
    e = torch.where(big <= LARGEST[fmt] * _two(e - 1), e - 1, e)
    scale = _two(e.clamp(LOWEST, HIGHEST[fmt]))
    z = z / scale[:, :, None]
    if fmt == "int8":
        step = torch.ones_like(z)
    else:
        step = _two(torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6))) - 3)   # 3 bits after the point
    z = (torch.round(z / step) * step).clamp(-LARGEST[fmt], LARGEST[fmt])
    return z.view(rows, n * GROUP)[:, :cols], scale


def _number64(held, cols, fmt):
    q, b = held
    n = -(-cols // GROUP)
    if fmt == "int8":
        v = q[:, :cols].to(torch.float64)
        v = torch.where(v > 127, v - 256, v)
    else:
        k = q[:, :cols].to(torch.int64)
        top, low = (k >> 3) & 15, (k & 7).double()
        v = torch.where(top > 0, (1 + low / 8) * _two(top - 7), low * 2.0 ** -9)
        v = torch.where(k >= 128, -v, v)
    exps = b[:, :n].double() - 127
    at = torch.div(torch.arange(cols, device=q.device), GROUP, rounding_mode="floor")
    return v * _two(exps)[:, at]


def exact(case, seed):
    s = prepare(case, seed)
    op, fmt = case["op"], case["fmt"]
    if op == "wgrad":
        n, m = case["n"], case["m"]
        x, dy = _number64(s["x8"], n, fmt), s["dy"].double()
        if case["groups"]:
            edges = _lengths(case["rows"], case["groups"], seed)
            g = torch.stack([dy[a:b].t().matmul(x[a:b]) for a, b in zip(edges, edges[1:])])
        else:
            g = dy.t().matmul(x)
        if case["scaled"]:
            g *= s["scale"].double()
        if case["accumulate"]:
            g += s["grad"].double()
        return {"grad": g}
    c = case["cols"]
    if op == "norm_fwd":
        h = s["x"].double() + (s["residual"].double() if case["residual"] else 0)
        r = 1 / torch.sqrt((h * h).sum(1) / c + EPS)
        n = h * r[:, None]
        y = n * s["weight"].double()
        q, sc = _round64(y if case["weighted"] else n, fmt)
        return {"h": h if case["residual"] else None, "y": y, "rstd": r, "saved": {"codes": q, "scales": sc}}
    if op == "norm_bwd":
        r = s["rstd"].double()[:, None]
        n = _number64(s["saved"], c, fmt) if case["from8"] else s["h"].double() * r
        dy = s["dy"].double()
        a = dy * s["weight"].double()
        dx = r * (a - n * ((a * n).sum(1, keepdim=True) / c))
        if case["residual"]:
            dx += s["dres"].double()
        return {"dx": dx, "dweight": (dy * n).sum(0)}
    if op == "glu_fwd":
        g, u = s["gu"][:, :c].double(), s["gu"][:, c:].double()
        a = g * u / (1 + torch.exp(-g))
        (gq, gs), (uq, us) = _round64(g, fmt), _round64(u, fmt)
        return {"a": a, "gate": {"codes": gq, "scales": gs}, "up": {"codes": uq, "scales": us}}
    if op == "glu_bwd":
        g, u, da = _number64(s["g8"], c, fmt), _number64(s["u8"], c, fmt), s["da"].double()
        p = 1 / (1 + torch.exp(-g))
        out = torch.cat([da * u * p * (1 + g * (1 - p)), da * g * p], dim=1)
        q, sc = _round64(g * p * u, fmt)
        return {"dgu": out, "a": {"codes": q, "scales": sc}}
    q, sc = _round64(s["wide"][:, 32:32 + c].double(), fmt)
    at = torch.div(torch.arange(c, device="cuda"), GROUP, rounding_mode="floor")
    return {"back": q * sc[:, at]}

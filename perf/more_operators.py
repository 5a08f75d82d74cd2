"""Cases of the operators around experts' weights on their way to the optimizer step:
tokens put in the experts' order and back (order, dispatch, combine), the experts'
products (forward and input gradient), and the global norm and clipping of the gradients.

``run`` computes an operator in its plain form (elementary torch operations in 32
bits, rounded once at the end), or, where ``own`` is true, through the framework's
entry points.  ``exact`` gives the same outputs from the definitions in 64 bits.

Experts' tokens are ranges of rows: expert e has rows offsets[e] .. offsets[e + 1] - 1.
slots[t, j] is the row that token t's choice j stands in, -1 where it chose no expert.
"""
import math
import random

import torch

own = False

_kept = {}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # decoding: eight rows, spread over 32 experts, most of whose weights are not touched
        {"name": "product_decode", "op": "product", "rows": 8, "m": 1024, "n": 2048, "groups": 32, "dgrad": False},
        # a short batch through a small weight with odd sides: rows without alignment
        {"name": "product_odd", "op": "product", "rows": 257, "m": 515, "n": 1001, "groups": 0, "dgrad": False},
        # 32 experts over 16k rows of ragged lengths, some without a row: their first product
        {"name": "product_experts", "op": "product", "rows": 16384, "m": 1024, "n": 2048, "groups": 32, "dgrad": False},
        # the gradient of its input
        {"name": "dgrad_experts", "op": "product", "rows": 16384, "m": 1024, "n": 2048, "groups": 32, "dgrad": True},
        # eight wide experts, an FFN of 18944 at hidden 3584, over 16k rows
        {"name": "product_ffn", "op": "product", "rows": 16384, "m": 18944, "n": 3584, "groups": 8, "dgrad": False},
        # the order of a small serving batch: latency alone
        {"name": "order_small", "op": "order", "tokens": 64, "choices": 8, "experts": 32},
        # the order of a training micro-batch, eight choices among 128 experts
        {"name": "order_16k", "op": "order", "tokens": 16384, "choices": 8, "experts": 128},
        # the micro-batch's rows put in the experts' order
        {"name": "dispatch_8k", "op": "dispatch", "tokens": 8192, "choices": 4, "experts": 32, "cols": 3584,
         "dtype": "bf16"},
        # a few tokens' rows of odd width in fp32, weighted and summed
        {"name": "combine_odd", "op": "combine", "tokens": 333, "choices": 3, "experts": 16, "cols": 1001,
         "dtype": "f32", "weighted": True},
        # the gradients of the weighted sum: the experts' rows and the router's weights
        {"name": "combine_bwd_8k", "op": "combine_bwd", "tokens": 8192, "choices": 4, "experts": 32, "cols": 3584,
         "dtype": "bf16"},
        # the gradients of one 7B decoder layer, fp32 sums of micro-batches, clipped into the bf16 that the step reads
        {"name": "clip_layer", "op": "clip", "layers": 1, "count": 0, "largest": 0, "dtype": "f32", "out": "bf16",
         "max_norm": 1.0, "salt": 0},
        # the norm alone over a thousand matrices of one model split per head, 128 x 3584 and smaller, in bf16
        {"name": "norm_heads", "op": "clip", "layers": 0, "count": 1036, "largest": 458752, "dtype": "bf16", "out": "",
         "max_norm": 1.0, "salt": 1},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], even over the logarithm; half of them odd as drawn, half rounded to 64."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if rng.random() < 0.5 and v >= 64:
        v = (v + 32) // 64 * 64
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["product", "product", "product", "order", "dispatch", "combine", "combine_bwd", "clip", "clip"])
    if op == "product":
        groups = rng.choice([0, _spread(rng, 2, 64), _spread(rng, 2, 64)])
        top = 4096 if groups else 8192
        return {"op": op, "rows": _spread(rng, 1, 16384), "m": _spread(rng, 128, top), "n": _spread(rng, 128, top),
                "groups": groups, "dgrad": rng.random() < 0.5}
    if op == "clip":
        dtype = rng.choice(["bf16", "f32"])
        # small gradients and few of them, up to hundreds of matrices
        count = _spread(rng, 1, 512)
        return {"op": op, "layers": 0, "count": count, "largest": _spread(rng, 1000, min(1 << 24, (1 << 28) // count)),
                "dtype": dtype, "out": rng.choice(["", "bf16", "f32"]), "max_norm": rng.choice([0.25, 1.0, 100.0]),
                "salt": rng.randrange(1 << 20)}
    case = {"op": op, "tokens": _spread(rng, 1, 32768), "choices": rng.randint(1, 8), "experts": _spread(rng, 2, 256)}
    if op == "order":
        return case
    case["cols"] = _spread(rng, 32, 8192)
    case["dtype"] = rng.choice(["bf16", "bf16", "f32"])
    case["tokens"] = max(1, min(case["tokens"], 117_000_000 // (case["cols"] * case["choices"])))
    if op == "combine":
        case["weighted"] = rng.random() < 0.7
    return case


def work(case):
    op = case["op"]
    if op == "product":
        t, m, n = case["rows"], case["m"], case["n"]
        lengths = [b - a for a, b in _pairs(_edges(t, case["groups"], 0))] if case["groups"] else [t]
        used, live = sum(lengths), sum(1 for x in lengths if x)
        return {"bytes": 2.0 * (used * (m + n) + live * m * n), "flops": 2.0 * used * m * n}
    if op == "clip":
        total, vectors = sum(s for s, v in _sizes(case) if not v), sum(s for s, v in _sizes(case) if v)
        e = 2 if case["dtype"] == "bf16" else 4
        out = {"": 0, "bf16": 2, "f32": 4}[case["out"]]
        # the norm has to have seen every value before the first can be scaled: they are read twice
        passes = 2 if case["out"] else 1
        return {"bytes": float(passes * (total * e + vectors * 4) + (total * out + (vectors * 4 if out else 0))),
                "flops": (2.0 + (1 if out else 0)) * (total + vectors)}
    t, k = case["tokens"], case["choices"]
    if op == "order":
        return {"bytes": 8.0 * t * k + 4 * (case["experts"] + 1), "flops": 1.0 * t * k}
    row = case["cols"] * (2 if case["dtype"] == "bf16" else 4)
    if op == "dispatch":
        return {"bytes": float(t * row * (1 + k) + 4 * t * k), "flops": 0.0}
    if op == "combine":
        return {"bytes": float(t * row * (1 + k) + (8 if case["weighted"] else 4) * t * k),
                "flops": 2.0 * t * k * case["cols"]}
    return {"bytes": float(t * row * (1 + 2 * k) + 12 * t * k), "flops": 3.0 * t * k * case["cols"]}


# ---------------------------------------------------------------- inputs
def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 64 + salt)
    return g


def _dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def _pairs(edges):
    return list(zip(edges, edges[1:]))


def _edges(rows, groups, seed):
    """Edges of the experts' ranges: uneven shares, about one expert in eight without a row; of long batches the last
    rows pad the batch and belong to none."""
    r = random.Random(seed)
    share = [0.0 if r.random() < 0.125 else r.expovariate(1.0) + 0.05 for _ in range(groups)]
    if not any(share):
        share[0] = 1.0
    used = rows - rows // 100
    edges, acc, total = [0], 0.0, sum(share)
    for x in share:
        acc += x
        edges.append(int(round(used * acc / total)))
    edges[-1] = used
    return edges


def _sizes(case):
    """(elements, is a vector) of each gradient: vectors (norm weights) are fp32 whatever the matrices are."""
    if case["layers"]:
        h, f, kv = 3584, 18944, 512
        one = [(h * h, False), (kv * h, False), (kv * h, False), (h * h, False), (f * h, False), (f * h, False),
               (h * f, False), (h, True), (h, True)]
        return one * case["layers"]
    r = random.Random(case["salt"])
    out = []
    for i in range(case["count"]):
        s = int(case["largest"] * math.exp(-1.5 * r.random())) if i else case["largest"]
        out.append((max(1, s), False) if r.random() < 0.9 or i == 0 else (max(1, min(s, 1 + s % 4096)), True))
    return out


def _activation(rows, cols, seed, salt, dtype):
    """Activations: a few channels far larger than the rest, tokens of unequal size."""
    g = _gen(seed, salt)
    x = torch.randn((rows, cols), generator=g, device="cuda")
    channel = torch.exp(0.5 * torch.randn((1, cols), generator=g, device="cuda"))
    channel = torch.where(torch.rand((1, cols), generator=g, device="cuda") < 0.002, 20.0 * channel, channel)
    return (x * channel * torch.exp(0.3 * torch.randn((rows, 1), generator=g, device="cuda"))).to(dtype)


def _gradient(rows, cols, seed, salt, dtype, scale=1e-2):
    g = _gen(seed, salt)
    x = torch.randn((rows, cols), generator=g, device="cuda")
    return (x * torch.exp(0.5 * torch.randn((rows, 1), generator=g, device="cuda")) * scale).to(dtype)


def _choices(case, seed):
    """Each token's experts, distinct, some experts far more wanted than others; about one token in a hundred pads
    the batch and chooses none."""
    t, k, e = case["tokens"], case["choices"], case["experts"]
    g = _gen(seed, 7)
    score = torch.rand((t, e), generator=g, device="cuda").log().neg()
    score = score * torch.exp(torch.randn((1, e), generator=g, device="cuda"))
    if k > e:
        ids = torch.randint(0, e, (t, k), generator=g, device="cuda")
    else:
        ids = score.topk(k, dim=1, largest=False).indices
    if t >= 16:
        ids = torch.where(torch.rand((t, 1), generator=g, device="cuda") < 0.01, torch.full_like(ids, -1), ids)
    return ids.to(torch.int32)


def _place(ids, experts):
    """(offsets, slots) of the stable order by expert, as the order operator gives them."""
    flat = ids.reshape(-1).long()
    key = torch.where(flat < 0, torch.full_like(flat, experts), flat)
    by = torch.argsort(key, stable=True)
    slots = torch.empty_like(by)
    slots[by] = torch.arange(by.numel(), device=by.device)
    slots = torch.where(flat < 0, torch.full_like(slots, -1), slots)
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device=by.device)
    offsets[1:] = torch.cumsum((flat[:, None] == torch.arange(experts, device=by.device)).sum(0), 0)
    return offsets, slots.reshape(ids.shape).to(torch.int32)


def prepare(case, seed):
    op = case["op"]
    s = {"case": case}
    if own:
        import matrix_orthogonalising_optimizer_muon_gb300 as muon
        if "plan" not in _kept:
            _kept["plan"] = muon.GradPlan()      # one plan serves every call of a program
        s["muon"], s["plan"] = muon, _kept["plan"]
    if op == "product":
        t, m, n, groups = case["rows"], case["m"], case["n"], case["groups"]
        k_in, k_out = (m, n) if case["dgrad"] else (n, m)
        s["x"] = (_gradient if case["dgrad"] else _activation)(t, k_in, seed, 1, torch.bfloat16)
        w = torch.empty((max(1, groups), m, n), dtype=torch.bfloat16, device="cuda")
        g = _gen(seed, 2)
        for e in range(w.shape[0]):
            w[e] = torch.randn((m, n), generator=g, device="cuda") * 0.02
        s["w"] = w if groups else w[0]
        s["out"] = torch.zeros((t, k_out), dtype=torch.bfloat16, device="cuda")
        # lengths are the case's, so that every seed is the same work; the host has them for the plain form alone
        s["edges"] = _edges(t, groups, 0) if groups else [0, t]
        s["offsets"] = torch.tensor(s["edges"], dtype=torch.int32, device="cuda") if groups else None
        return s
    if op == "clip":
        s["grads"], s["out"] = [], []
        g = _gen(seed, 3)
        for size, vector in _sizes(case):
            x = torch.empty((size,), dtype=torch.float32 if vector else _dt(case["dtype"]), device="cuda")
            x.copy_(torch.randn((size,), generator=g, device="cuda"))
            x *= 1e-3 * math.exp(random.Random(seed * 4096 + size).gauss(0, 0.5))
            s["grads"].append(x)
            if case["out"]:
                s["out"].append(torch.empty((size,), dtype=torch.float32 if vector else _dt(case["out"]),
                                            device="cuda"))
        s["norm"] = torch.zeros((1,), device="cuda")
        if own:
            s["grad_list"] = s["muon"].GradList(s["grads"])
            s["out_list"] = s["muon"].GradList(s["out"]) if case["out"] else None
        return s
    s["ids"] = _choices(case, seed)
    if op == "order":
        s["offsets"] = torch.empty((case["experts"] + 1,), dtype=torch.int32, device="cuda")
        s["slots"] = torch.empty_like(s["ids"])
        return s
    t, k, c, dt = case["tokens"], case["choices"], case["cols"], _dt(case["dtype"])
    s["slots"] = _place(s["ids"], case["experts"])[1]
    s["weights"] = torch.softmax(torch.randn((t, k), generator=_gen(seed, 4), device="cuda"), 1)
    if op == "dispatch":
        s["x"] = _activation(t, c, seed, 1, dt)
        s["out"] = torch.zeros((t * k, c), dtype=dt, device="cuda")
        return s
    s["rows"] = _activation(t * k, c, seed, 1, dt)
    if op == "combine":
        s["out"] = torch.zeros((t, c), dtype=dt, device="cuda")
        if not case["weighted"]:
            s["weights"] = None
        return s
    s["dout"] = _gradient(t, c, seed, 5, dt)
    s["drows"] = torch.zeros_like(s["rows"])
    s["dweights"] = torch.zeros_like(s["weights"])
    return s


# ---------------------------------------------------------------- plain forms
def _plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "product":
        for e, (a, b) in enumerate(_pairs(s["edges"])):
            if a < b:
                w = (s["w"][e] if case["groups"] else s["w"]).float()
                s["out"][a:b] = s["x"][a:b].float() @ (w if case["dgrad"] else w.t())
        return {"out": s["out"]}
    if op == "clip":
        total = torch.stack([g.float().square().sum(dtype=torch.float64) for g in s["grads"]]).sum()
        norm = total.sqrt()
        s["norm"][0] = norm
        if not case["out"]:
            return {"norm": s["norm"]}
        # the factor in 32 bits from the rounded norm, as an operator that is handed the norm has it
        factor = torch.where(s["norm"] > case["max_norm"], case["max_norm"] / s["norm"], torch.ones_like(s["norm"]))
        for o, g in zip(s["out"], s["grads"]):
            o.copy_(g.float() * factor)
        return {"norm": s["norm"], "out": s["out"]}
    if op == "order":
        offsets, slots = _place(s["ids"], case["experts"])
        s["offsets"].copy_(offsets)
        s["slots"].copy_(slots)
        return {"offsets": s["offsets"], "slots": s["slots"]}
    slots = s["slots"].long()
    there = slots >= 0
    at = slots.clamp(min=0)
    if op == "dispatch":
        for j in range(case["choices"]):
            have = there[:, j]
            s["out"][at[have, j]] = s["x"][have]
        return {"out": s["out"]}
    if op == "combine":
        acc = torch.zeros(s["out"].shape, device="cuda")
        for j in range(case["choices"]):
            v = s["rows"][at[:, j]].float()
            if s["weights"] is not None:
                v = v * s["weights"][:, j, None]
            acc += torch.where(there[:, j, None], v, torch.zeros_like(v))
        s["out"].copy_(acc)
        return {"out": s["out"]}
    dout = s["dout"].float()
    for j in range(case["choices"]):
        have = there[:, j]
        s["drows"][at[have, j]] = (s["weights"][have, j, None] * dout[have]).to(s["drows"].dtype)
        dot = (dout * s["rows"][at[:, j]].float()).sum(1)
        s["dweights"][:, j] = torch.where(have, dot, torch.zeros_like(dot))
    return {"drows": s["drows"], "dweights": s["dweights"]}


# ---------------------------------------------------------------- the framework's calls
def _own(s):
    case, muon, plan = s["case"], s["muon"], s["plan"]
    op = case["op"]
    if op == "product":
        (plan.dgrad if case["dgrad"] else plan.product)(s["x"], s["w"], s["out"], offsets=s["offsets"])
        return {"out": s["out"]}
    if op == "clip":
        plan.grad_norm(s["grad_list"], s["norm"])
        if not case["out"]:
            return {"norm": s["norm"]}
        plan.grad_clip(s["grad_list"], s["norm"], case["max_norm"], out=s["out_list"])
        return {"norm": s["norm"], "out": s["out"]}
    if op == "order":
        muon.expert_order(s["ids"], s["offsets"], s["slots"])
        return {"offsets": s["offsets"], "slots": s["slots"]}
    if op == "dispatch":
        muon.expert_dispatch(s["x"], s["slots"], s["out"])
        return {"out": s["out"]}
    if op == "combine":
        muon.expert_combine(s["rows"], s["slots"], s["out"], weights=s["weights"])
        return {"out": s["out"]}
    muon.expert_combine_backward(s["dout"], s["slots"], s["weights"], rows=s["rows"], drows=s["drows"],
                                 dweights=s["dweights"])
    return {"drows": s["drows"], "dweights": s["dweights"]}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- definitions in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "product":
        if 2.0 * case["rows"] * case["m"] * case["n"] > 5e12:
            return None
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        ends = s["edges"]
        for e in range(len(ends) - 1):
            w = s["w"].reshape(-1, case["m"], case["n"])[e]
            rows = s["x"][ends[e]:ends[e + 1]].double()
            eq = "tm,mn->tn" if case["dgrad"] else "tn,mn->tm"
            if rows.shape[0]:
                out[ends[e]:ends[e + 1]] = torch.einsum(eq, rows, w.double())
        return {"out": out}
    if op == "clip":
        total = sum((torch.dot(g.double(), g.double()) for g in s["grads"]),
                    torch.zeros((), dtype=torch.float64, device="cuda"))
        norm = float(total) ** 0.5
        if not case["out"]:
            return {"norm": torch.tensor([norm], dtype=torch.float64, device="cuda")}
        factor = min(1.0, case["max_norm"] / norm) if norm > 0 else 1.0
        return {"norm": torch.tensor([norm], dtype=torch.float64, device="cuda"),
                "out": [g.double() * factor for g in s["grads"]]}
    if op == "order":
        ids = s["ids"].cpu().reshape(-1).tolist()
        lists = [[] for _ in range(case["experts"])]
        for i, e in enumerate(ids):
            if 0 <= e < case["experts"]:
                lists[e].append(i)
        offsets, slots = [0], [-1] * len(ids)
        for places in lists:
            for j, i in enumerate(places):
                slots[i] = offsets[-1] + j
            offsets.append(offsets[-1] + len(places))
        return {"offsets": torch.tensor(offsets, device="cuda"),
                "slots": torch.tensor(slots, device="cuda").reshape(s["ids"].shape)}
    slots = s["slots"].reshape(-1).long()
    flat = torch.nonzero(slots >= 0).reshape(-1)                  # (token, choice) pairs that stand somewhere
    where, token = slots[flat], flat // case["choices"]
    if op == "dispatch":
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        out.index_copy_(0, where, s["x"].double().index_select(0, token))
        return {"out": out}
    weight = torch.ones(slots.shape, dtype=torch.float64, device="cuda")
    if s["weights"] is not None:
        weight = s["weights"].double().reshape(-1)
    if op == "combine":
        out = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
        out.index_add_(0, token, s["rows"].double().index_select(0, where) * weight[flat][:, None])
        return {"out": out}
    dout = s["dout"].double().index_select(0, token)
    drows = torch.zeros(s["drows"].shape, dtype=torch.float64, device="cuda")
    drows.index_copy_(0, where, dout * weight[flat][:, None])
    dweights = torch.zeros(slots.shape, dtype=torch.float64, device="cuda")
    dweights[flat] = torch.einsum("rc,rc->r", dout, s["rows"].double().index_select(0, where))
    return {"drows": drows, "dweights": dweights.reshape(s["weights"].shape)}

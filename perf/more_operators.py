"""Timed cases of the bf16 products and of what groups them by expert: the dense
product with its epilogue, the sort of routes by expert, the products over ragged
groups, and the weighted sum of a row's routes.

A case is a dict of plain values.  ``prepare`` makes what a serving program has
in hand before the call, ``run`` makes one pass, either in plain torch
operations in 32 bits (``own`` false) or through the library (``own`` true),
and ``exact`` gives the same outputs from the definitions in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

DEV = "cuda"
BF16 = torch.bfloat16


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # one token through a square projection, added to the bf16 residual stream
        dict(name="linear_token", op="linear", rows=1, n=4096, k=4096, act="none", gated=False,
             bias=False, res=True, out="bf16", alpha=1.0),
        # a wide decode step's dense expert: gate and up in one product (2 x 768)
        dict(name="linear_wide", op="linear", rows=600, n=768, k=2048, act="silu", gated=True,
             bias=False, res=False, out="bf16", alpha=1.0),
        # sizes that fill no tile, an fp32 residual stream, a bias and a residual multiplier
        dict(name="linear_ragged", op="linear", rows=1333, n=1001, k=2072, act="gelu", gated=False,
             bias=True, res=True, out="f32", alpha=0.22),
        # a prefill chunk through a dense projection
        dict(name="linear_prefill", op="linear", rows=8192, n=8192, k=4096, act="gelu_tanh",
             gated=False, bias=True, res=True, out="bf16", alpha=1.0),
        # one token's eight routes over 256 experts
        dict(name="group_token", op="group", rows=1, top=8, experts=256, dropped=0.0),
        # a prefill chunk's 65,536 routes, some without a slot
        dict(name="group_prefill", op="group", rows=8192, top=8, experts=256, dropped=0.05),
        # one token: the gate and up products of its eight experts
        dict(name="experts_token", op="experts", rows=1, top=8, experts=256, n=512, k=2048,
             gather=True, act="silu", gated=True, bias=False, out="bf16", dropped=0.0),
        # a wide decode step over 1,024 experts: one or two rows for most, their weights' bytes count
        dict(name="experts_wide", op="experts", rows=600, top=2, experts=1024, n=768, k=2048,
             gather=True, act="silu", gated=True, bias=False, out="bf16", dropped=0.1),
        # a prefill chunk: gate and up products, a few hundred rows for each of 256 experts
        dict(name="experts_prefill", op="experts", rows=8192, top=8, experts=256, n=512, k=2048,
             gather=True, act="silu", gated=True, bias=False, out="bf16", dropped=0.0),
        # the down products of the larger experts' chunk
        dict(name="experts_down", op="experts", rows=4096, top=8, experts=256, n=4096, k=1024,
             gather=False, act="none", gated=False, bias=False, out="bf16", dropped=0.05),
        # one token's eight routes back into its row
        dict(name="combine_token", op="combine", rows=1, top=8, experts=256, hidden=2048,
             y="bf16", add=True, out="bf16", dropped=0.0),
        # a prefill chunk's, beside the dense expert's output
        dict(name="combine_prefill", op="combine", rows=8192, top=8, experts=256, hidden=2048,
             y="bf16", add=True, out="bf16", dropped=0.05),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi, step):
    """A multiple of step spread over [lo, hi]'s logarithm."""
    return max(lo, min(hi, _log(rng, lo, hi) // step * step))


ACTS = ("none", "silu", "gelu", "gelu_tanh", "relu")


def draw(rng):
    op = rng.choice(("linear", "linear", "group", "experts", "experts", "combine"))
    out = rng.choice(("bf16", "f32"))
    if op == "linear":
        gated = rng.random() < 0.4
        k = _width(rng, 256, 8192, rng.choice((8, 64)))
        n = _width(rng, 256, 8192, rng.choice((1, 8, 64)) if not gated else 16)
        rows = _log(rng, 1, 8192)
        while rows * k * n * (1 + gated) > 8192 * 8192 * 4096:
            rows = max(1, rows // 2)
        return dict(op=op, rows=rows, n=n, k=k, act=rng.choice(ACTS), gated=gated,
                    bias=rng.random() < 0.5, res=rng.random() < 0.5, out=out,
                    alpha=rng.choice((1.0, 0.22)))
    experts = rng.choice((8, 16, 60, 64, 128, 160, 256, 384, 512, 1000, 1024))
    rows, top = _log(rng, 1, 8192), rng.choice((1, 2, 4, 6, 8))
    dropped = rng.choice((0.0, 0.0, 0.05, 0.3))
    if op == "group":
        return dict(op=op, rows=rows, top=top, experts=experts, dropped=dropped)
    if op == "combine":
        hidden = _width(rng, 512, 4096, rng.choice((1, 8, 64)))
        rows = min(rows, 8192 * 8 * 2048 // (hidden * top) // (1 if out == "bf16" else 2))
        return dict(op=op, rows=rows, top=top, experts=experts, hidden=hidden,
                    y=rng.choice(("bf16", "f32")) if out == "f32" else "bf16",
                    add=rng.random() < 0.5, out=out, dropped=dropped)
    gated = rng.random() < 0.5
    k = _width(rng, 256, 4096, rng.choice((8, 64)))
    n = _width(rng, 256, 4096, 16 if gated else rng.choice((1, 8, 64)))
    while experts * n * k * (1 + gated) > 1024 * 768 * 2048 * 2:
        n = max(256, n // 2 // 16 * 16)
        k = max(256, k // 2 // 8 * 8)
    while rows * top * n * k * (1 + gated) > 8192 * 8 * 1024 * 2048:
        rows = max(1, rows // 2)
    return dict(op=op, rows=rows, top=top, experts=experts, n=n, k=k, gather=rng.random() < 0.5,
                act=rng.choice(ACTS), gated=gated, bias=rng.random() < 0.3, out=out, dropped=dropped)


# ------------------------------------------------------------------- the inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _normal(g, *shape, std=1.0, dtype=BF16):
    return torch.randn(*shape, generator=g, device=DEV, dtype=dtype).mul_(std)


def _dtype(name):
    return BF16 if name == "bf16" else torch.float32


def prepare(case, seed):
    g = _gen(seed)
    return {"linear": _prepare_linear, "group": _prepare_group, "experts": _prepare_experts,
            "combine": _prepare_combine}[case["op"]](case, g)


def _prepare_linear(c, g):
    B, N, K = c["rows"], c["n"], c["k"]
    wide = N * (1 + c["gated"])
    s = dict(c, x=_normal(g, B, K), w=_normal(g, wide, K, std=K ** -0.5))
    s["b"] = _normal(g, wide, std=0.5) if c["bias"] else None
    s["r"] = _normal(g, B, N, std=4.0, dtype=_dtype(c["out"])) if c["res"] else None
    s["y"] = torch.empty(B, N, dtype=_dtype(c["out"]), device=DEV)
    return s


def _routes(c, g):
    """int32 [rows][top]: distinct experts of uneven popularity, some routes without one."""
    B, E, k = c["rows"], c["experts"], c["top"]
    z = torch.randn(B, E, generator=g, device=DEV) + 0.7 * torch.randn(E, generator=g, device=DEV)
    ids = z.topk(k, 1).indices.to(torch.int32)
    gone = torch.rand(B, k, generator=g, device=DEV) < c["dropped"]
    return ids.masked_fill(gone, -1)


def _grouped(ids, E):
    """(offsets [E + 1], order, pos): the routes by (expert, route); -1 for what has no place."""
    flat = ids.reshape(-1)
    R = flat.numel()
    ok = (flat >= 0) & (flat < E)
    key = torch.where(ok, flat, E).long()
    order = key.sort(stable=True).indices
    count = torch.zeros(E + 1, dtype=torch.long, device=DEV).index_add_(0, key, torch.ones_like(key))
    offsets = torch.cat((count.new_zeros(1), count[:E].cumsum(0)))
    place = torch.arange(R, device=DEV)
    pos = torch.empty_like(place).scatter_(0, order, place)
    pos = torch.where(ok, pos, -1)
    order = torch.where(place < offsets[E], order, -1)
    i32 = torch.int32
    return offsets.to(i32), order.to(i32), pos.to(i32)


def _prepare_group(c, g):
    R, i32 = c["rows"] * c["top"], torch.int32
    return dict(c, ids=_routes(c, g), offsets=torch.empty(c["experts"] + 1, dtype=i32, device=DEV),
                order=torch.empty(R, dtype=i32, device=DEV), pos=torch.empty(R, dtype=i32, device=DEV))


def _prepare_experts(c, g):
    E, N, K = c["experts"], c["n"], c["k"]
    wide = N * (1 + c["gated"])
    ids = _routes(c, g)
    offsets, order, _ = _grouped(ids, E)
    R = ids.numel()
    s = dict(c, offsets=offsets, order=order, x=_normal(g, c["rows"] if c["gather"] else R, K))
    s["w"] = _normal(g, E, wide, K, std=K ** -0.5)
    s["b"] = _normal(g, E, wide, std=0.5) if c["bias"] else None
    s["starts"] = offsets.tolist()          # the plain form's loop runs on the host
    # rows without a place stay as they were
    s["y"] = torch.zeros(R, N, dtype=_dtype(c["out"]), device=DEV)
    return s


def _prepare_combine(c, g):
    ids = _routes(c, g)
    _, _, pos = _grouped(ids, c["experts"])
    H, out = c["hidden"], _dtype(c["out"])
    s = dict(c, posv=pos.reshape(ids.shape), yv=_normal(g, ids.numel(), H, dtype=_dtype(c["y"])))
    s["w"] = torch.rand(*ids.shape, generator=g, device=DEV)
    s["w"] /= s["w"].sum(1, keepdim=True)
    s["addv"] = _normal(g, c["rows"], H, dtype=out) if c["add"] else None
    s["o"] = torch.empty(c["rows"], H, dtype=out, device=DEV)
    return s


# ------------------------------------------------------------------- one pass

def run(s):
    return (_OWN if own else _PLAIN)[s["op"]](s)


def _lib():
    import expert_slot_cache_lru_gb300 as m
    return m


def _act_id(m, name):
    return {"none": m.MOE_ACT_NONE, "silu": m.MOE_ACT_SILU, "gelu": m.MOE_ACT_GELU,
            "gelu_tanh": m.MOE_ACT_GELU_TANH, "relu": m.MOE_ACT_RELU}[name]


def _own_linear(s):
    m = _lib()
    m.moe_linear(s["x"], s["w"], s["b"], s["r"], s["y"], s["rows"], s["n"], s["k"],
                 act=_act_id(m, s["act"]), gated=s["gated"], alpha=s["alpha"],
                 dtype=m.MOE_T_BF16 if s["out"] == "bf16" else m.MOE_T_F32)
    return s["y"]


def _own_group(s):
    m = _lib()
    m.moe_group_routes(s["ids"], s["rows"] * s["top"], s["experts"], s["offsets"], s["order"], s["pos"])
    return s["offsets"], s["order"], s["pos"]


def _own_experts(s):
    m = _lib()
    m.moe_grouped_linear(s["x"], s["x"].shape[0], s["order"] if s["gather"] else None, s["top"],
                         s["offsets"], s["experts"], s["w"], s["b"], s["y"], s["y"].shape[0], s["n"],
                         s["k"], act=_act_id(m, s["act"]), gated=s["gated"],
                         dtype=m.MOE_T_BF16 if s["out"] == "bf16" else m.MOE_T_F32)
    return s["y"]


def _own_combine(s):
    m = _lib()
    t = {"bf16": m.MOE_T_BF16, "f32": m.MOE_T_F32}
    m.moe_combine(s["yv"], s["yv"].shape[0], s["posv"], s["w"], s["addv"], s["o"], s["rows"], s["top"],
                  s["hidden"], y_dtype=t[s["y"]], dtype=t[s["out"]])
    return s["o"]


def _act(z, kind):
    if kind == "silu":
        return z / (1 + torch.exp(-z))
    if kind == "gelu":
        return z * 0.5 * torch.erfc(-z * 0.7071067811865476)
    if kind == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(0.7978845608028654 * (z + 0.044715 * z * z * z)))
    return torch.clamp(z, min=0.0) if kind == "relu" else z


def _plain_product(x, w, b, s):
    z = x.float() @ w.float().T
    if b is not None:
        z = z + b.float()
    if s["gated"]:
        return _act(z[:, :s["n"]], s["act"]) * z[:, s["n"]:]
    return _act(z, s["act"])


def _plain_linear(s):
    y = s["alpha"] * _plain_product(s["x"], s["w"], s["b"], s)
    if s["r"] is not None:
        y = s["r"].float() + y
    return y.to(s["y"].dtype)


def _plain_group(s):
    return _grouped(s["ids"], s["experts"])


def _plain_experts(s):
    at, y = s["starts"], s["y"]
    rows = (s["order"] // s["top"]).long() if s["gather"] else None
    for e in range(s["experts"]):
        lo, hi = at[e], at[e + 1]
        if lo < hi:
            x = s["x"][rows[lo:hi]] if s["gather"] else s["x"][lo:hi]
            y[lo:hi] = _plain_product(x, s["w"][e], s["b"][e] if s["b"] is not None else None, s)
    return y


def _plain_combine(s):
    placed = s["posv"] >= 0
    acc = s["addv"].float() if s["addv"] is not None else 0.0
    for j in range(s["top"]):
        y = s["yv"][s["posv"][:, j].clamp(min=0).long()].float() * s["w"][:, j:j + 1]
        acc = acc + torch.where(placed[:, j:j + 1], y, torch.zeros_like(y))
    return acc.to(s["o"].dtype)


_OWN = {"linear": _own_linear, "group": _own_group, "experts": _own_experts, "combine": _own_combine}
_PLAIN = {"linear": _plain_linear, "group": _plain_group, "experts": _plain_experts,
          "combine": _plain_combine}


# ------------------------------------------------------------------- the floor

def _filled(c):
    """Expected number of experts with a row, at even popularity."""
    E, R = c["experts"], c["rows"] * c["top"] * (1 - c["dropped"])
    return E * (1 - (1 - 1 / E) ** R)


def work(c):
    """Bytes read and written once and operations of one pass."""
    t = 2 if c.get("out") == "bf16" else 4
    if c["op"] == "linear":
        B, N, K, wide = c["rows"], c["n"], c["k"], c["n"] * (1 + c["gated"])
        return {"bytes": 2 * B * K + 2 * wide * K + B * N * t * (1 + c["res"]) + 2 * wide * c["bias"],
                "flops": 2 * B * wide * K}
    R = c["rows"] * c["top"]
    if c["op"] == "group":
        return {"bytes": 12 * R + 4 * (c["experts"] + 1), "flops": 4 * R}
    placed = R * (1 - c["dropped"])
    if c["op"] == "experts":
        N, K, wide = c["n"], c["k"], c["n"] * (1 + c["gated"])
        x = 2 * K * (c["rows"] if c["gather"] else placed) + (4 * placed if c["gather"] else 0)
        return {"bytes": int(x + 2 * _filled(c) * wide * (K + c["bias"]) + placed * N * t),
                "flops": int(2 * placed * wide * K)}
    H, ty = c["hidden"], 2 if c["y"] == "bf16" else 4
    return {"bytes": int(placed * H * ty + 8 * R + c["rows"] * H * t * (1 + c["add"])),
            "flops": int(2 * placed * H)}


# ------------------------------------------------------------------- 64 bits

def exact(case, seed):
    if case["op"] == "group":  # whole numbers, all of them
        return None
    s = prepare(case, seed)
    return {"linear": _exact_linear, "experts": _exact_experts, "combine": _exact_combine}[case["op"]](s)


def _exact_act(z, kind):
    if kind == "silu":
        return z * torch.special.expit(z)
    if kind == "gelu":
        return z * torch.special.ndtr(z)
    if kind == "gelu_tanh":
        # (1 + tanh u) / 2 is a sigmoid of 2 u
        return z * torch.special.expit(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return torch.where(z > 0, z, torch.zeros_like(z)) if kind == "relu" else z


def _exact_product(x, w, b, s):
    d = torch.float64
    z = torch.einsum("bk,nk->bn", x.to(d), w.to(d))
    if b is not None:
        z += b.to(d)
    if not s["gated"]:
        return _exact_act(z, s["act"])
    gate, up = z.split(s["n"], 1)
    return _exact_act(gate, s["act"]) * up


def _exact_linear(s):
    y = _exact_product(s["x"], s["w"], s["b"], s)
    return y.mul_(s["alpha"]) if s["r"] is None else torch.add(s["r"].double(), y, alpha=s["alpha"])


def _exact_experts(s):
    y = torch.zeros(s["y"].shape, dtype=torch.float64, device=DEV)
    counts = [b - a for a, b in zip(s["starts"], s["starts"][1:])]
    owner = torch.repeat_interleave(torch.arange(s["experts"], device=DEV), torch.tensor(counts, device=DEV))
    for e in range(s["experts"]):
        mine = (owner == e).nonzero().flatten()
        if mine.numel():
            src = torch.div(s["order"][mine], s["top"], rounding_mode="floor").long() if s["gather"] else mine
            y.index_copy_(0, mine, _exact_product(s["x"].index_select(0, src), s["w"][e],
                                                  None if s["b"] is None else s["b"][e], s))
    return y


def _exact_combine(s):
    B, k = s["posv"].shape
    o = torch.zeros(B, s["hidden"], dtype=torch.float64, device=DEV)
    if s["addv"] is not None:
        o += s["addv"]
    b, j = (s["posv"] >= 0).nonzero(as_tuple=True)
    step = 16384
    for i in range(0, b.numel(), step):
        bb, jj = b[i:i + step], j[i:i + step]
        o.index_add_(0, bb, s["yv"][s["posv"][bb, jj].long()].double() * s["w"][bb, jj].double().unsqueeze(1))
    return o

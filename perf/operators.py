"""Timed cases of the operators around the expert cache: the block norm, the
router, the 4-bit conversions and the 4-bit product.

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
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------- the cases

def listed():
    return [
        # one token through a decode layer: latency, both norms, bf16 residual
        dict(name="norm_decode", op="norm", rows=1, hidden=2048, res="bf16", post=True, gate="none",
             alpha=1.0, offset=0.0),
        # a wide decode step: fp32 residual stream, a sigmoid gate for each row
        dict(name="norm_wide", op="norm", rows=600, hidden=2048, res="f32", post=False,
             gate="sigmoid_rows", alpha=1.0, offset=0.0),
        # a prefill chunk: learned gate per channel, residual multiplier, 1 + w weights
        dict(name="norm_prefill", op="norm", rows=8192, hidden=4096, res="bf16", post=True,
             gate="channel", alpha=0.22, offset=1.0),
        # one token's router: 256 experts, top 8, renormalised softmax
        dict(name="route_decode", op="route", rows=1, hidden=2048, experts=256, k=8,
             score="softmax", bias=False, groups=1, topk_groups=1, group_top=1, renorm=True,
             scale=1.0),
        # the wide decode step: 600 rows, 1,024 experts, top 2, sigmoid scores with a balance bias
        dict(name="route_wide", op="route", rows=600, hidden=2048, experts=1024, k=2,
             score="sigmoid", bias=True, groups=1, topk_groups=1, group_top=1, renorm=True,
             scale=1.0),
        # a prefill chunk: grouped choice (4 of 8 groups by their two best), bias, scaled weights
        dict(name="route_prefill", op="route", rows=8192, hidden=4096, experts=256, k=8,
             score="sigmoid", bias=True, groups=8, topk_groups=4, group_top=2, renorm=True,
             scale=2.5),
        # a short chunk's activations through 4 bits
        dict(name="quantize_chunk", op="quantize", rows=64, cols=2048, fmt="nvfp4", src="bf16"),
        # a ragged fp32 matrix (rows and blocks that fill no tile) in the other format
        dict(name="quantize_ragged", op="quantize", rows=1333, cols=2080, fmt="mxfp4", src="f32"),
        # one projection of a layer's 256 experts (512 x 2,048 each) turned into 4 bits and checked
        dict(name="quantize_experts", op="quantize", rows=131072, cols=2048, fmt="nvfp4",
             src="bf16"),
        # one token's logits: the 4-bit head over 131,072 words
        dict(name="linear_token", op="linear", rows=1, k=2048, n=131072, fmt="nvfp4", out="f32"),
        # a wide decode step's gate and up projections of a dense expert (2 x 768)
        dict(name="linear_wide", op="linear", rows=600, k=2048, n=1536, fmt="mxfp4", out="bf16"),
        # a prefill chunk through a dense projection
        dict(name="linear_prefill", op="linear", rows=8192, k=4096, n=8192, fmt="nvfp4",
             out="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi, step):
    """A multiple of step spread over [lo, hi]'s logarithm."""
    w = max(lo, min(hi, _log(rng, lo, hi) // step * step))
    return w + step if w == 3072 else w


def draw(rng):
    op = rng.choice(("norm", "route", "quantize", "linear"))
    if op == "norm":
        hidden = _width(rng, 512, 8192, rng.choice((1, 8, 64)))
        return dict(op=op, rows=min(_log(rng, 1, 8192), 8192 * 4096 // hidden), hidden=hidden,
                    res=rng.choice(("bf16", "f32")), post=rng.random() < 0.5,
                    gate=rng.choice(("none", "channel", "sigmoid_rows")),
                    alpha=rng.choice((1.0, 0.22)), offset=rng.choice((0.0, 1.0)))
    if op == "route":
        groups = rng.choice((1, 1, 4, 8))
        experts = groups * rng.choice((16, 20, 32, 48, 64)) if groups > 1 else rng.choice(
            (16, 60, 64, 128, 160, 256, 384, 512, 1000, 1024))
        hidden = _width(rng, 512, 4096, rng.choice((8, 64)))
        rows = min(_log(rng, 1, 8192), 8192 * 256 // experts)
        return dict(op=op, rows=rows, hidden=hidden, experts=experts, k=rng.choice((1, 2, 4, 6, 8)),
                    score=rng.choice(("softmax", "sigmoid")), bias=rng.random() < 0.5,
                    groups=groups, topk_groups=max(1, groups // 2),
                    group_top=rng.choice((1, 2)) if groups > 1 else 1, renorm=rng.random() < 0.7,
                    scale=rng.choice((1.0, 2.5)))
    if op == "quantize":
        cols = _width(rng, 512, 8192, 32)
        return dict(op=op, rows=min(_log(rng, 1, 131072), 131072 * 1024 // cols), cols=cols,
                    fmt=rng.choice(("nvfp4", "mxfp4")), src=rng.choice(("bf16", "f32")))
    k = _width(rng, 512, 8192, 32)
    n = _log(rng, 512, 65536)
    n += n == 3072
    rows = _log(rng, 1, 8192)
    while rows * k * n > 8192 * 4096 * 4096:
        rows = max(1, rows // 2)
    while n * k > 131072 * 1024:
        n //= 2
    return dict(op=op, rows=rows, k=k, n=n, fmt=rng.choice(("nvfp4", "mxfp4")),
                out=rng.choice(("bf16", "f32")))


# ------------------------------------------------------------------- the inputs

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def _normal(g, *shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(*shape, generator=g, device=DEV) * std).to(dtype)


def _dtype(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def prepare(case, seed):
    g = _gen(seed)
    return {"norm": _prepare_norm, "route": _prepare_route, "quantize": _prepare_quantize,
            "linear": _prepare_linear}[case["op"]](case, g)


def _prepare_norm(c, g):
    B, H = c["rows"], c["hidden"]
    s = dict(c, h=_normal(g, B, H, std=4.0, dtype=_dtype(c["res"])), y=_normal(g, B, H))
    centre = 1.0 - c["offset"]
    s["pre_w"] = (centre + 0.1 * torch.randn(H, generator=g, device=DEV)).to(torch.bfloat16)
    s["post_w"] = ((centre + 0.1 * torch.randn(H, generator=g, device=DEV)).to(torch.bfloat16)
                   if c["post"] else None)
    s["gatev"] = {"none": lambda: None, "channel": lambda: _normal(g, H, std=0.5),
                  "sigmoid_rows": lambda: _normal(g, B, H)}[c["gate"]]()
    s["h_out"], s["x_out"] = torch.empty_like(s["h"]), torch.empty_like(s["y"])
    return s


def _prepare_route(c, g):
    B, H, E = c["rows"], c["hidden"], c["experts"]
    s = dict(c, router=_normal(g, E, H, std=H ** -0.5), x=_normal(g, B, H))
    # the balance bias moves in steps of 0.001
    s["biasv"] = (torch.randint(-60, 61, (E,), generator=g, device=DEV).float() * 0.001
                  if c["bias"] else None)
    # a choice closer than two summation orders differ has no single answer, and ids are compared
    # as whole numbers: such rows (about one in a thousand) are drawn again
    for _ in range(20):
        bad = _unclear(s).nonzero().flatten()
        if not bad.numel():
            break
        s["x"][bad] = _normal(g, bad.numel(), H)
    s["logits"] = torch.empty(B, E, device=DEV)
    s["ids"] = torch.empty(B, c["k"], dtype=torch.int32, device=DEV)
    s["w"] = torch.empty(B, c["k"], device=DEV)
    return s


def _unclear(s):
    """Rows whose ranking would change with an error of 1e-5 in a logit."""
    z = s["x"].double() @ s["router"].double().T
    sc, choice, eligible = _choice(s, z)
    # a logit's error reaches a softmax score times the score, a sigmoid's at a quarter at most
    width = 4e-5 if s["biasv"] is None else 1e-5
    top = choice.masked_fill(~eligible, -math.inf).sort(dim=1, descending=True).values[:, :s["k"] + 1]
    near = (top[:, :-1] - top[:, 1:] < width).any(1)
    if s["groups"] > 1:
        gs = _group_scores(s, sc, choice).sort(dim=1, descending=True).values
        cut = s["topk_groups"]
        near |= gs[:, cut - 1] - gs[:, cut] < width * (1 if s["biasv"] is not None else 0.05)
    return near


def _prepare_quantize(c, g):
    B, K = c["rows"], c["cols"]
    blk = 16 if c["fmt"] == "nvfp4" else 32
    src = _normal(g, B, K, std=0.02, dtype=_dtype(c["src"]))
    # the largest magnitude expected, over 448 * 6
    glob = torch.tensor([0.1137 / 2688.0], device=DEV) if c["fmt"] == "nvfp4" else None
    return dict(c, src_t=src, glob=glob,
                codes=torch.empty(B, K // 2, dtype=torch.uint8, device=DEV),
                scales=torch.empty(B, K // blk, dtype=torch.uint8, device=DEV),
                values=torch.empty(B, K, dtype=_dtype(c["src"]), device=DEV))


def _prepare_linear(c, g):
    B, K, N = c["rows"], c["k"], c["n"]
    nv = c["fmt"] == "nvfp4"
    blk = 16 if nv else 32
    x = torch.randn(B, K, generator=g, device=DEV)
    x[:, :: 97] *= 4.0  # outlier channels
    lo, hi = (0x28, 0x38) if nv else (118, 122)
    s = dict(c, x=x.to(torch.bfloat16),
             wc=torch.randint(0, 256, (N, K // 2), generator=g, device=DEV, dtype=torch.uint8),
             ws=torch.randint(lo, hi, (N, K // blk), generator=g, device=DEV, dtype=torch.uint8))
    s["xg"] = torch.tensor([15.37 / 2688.0], device=DEV) if nv else None  # from a calibration
    s["wg"] = torch.tensor([0.011], device=DEV) if nv else None
    s["xc"] = torch.empty(B, K // 2, dtype=torch.uint8, device=DEV)
    s["xs"] = torch.empty(B, K // blk, dtype=torch.uint8, device=DEV)
    s["y"] = torch.empty(B, N, dtype=_dtype(c["out"]), device=DEV)
    return s


# ------------------------------------------------------------------- one pass

def run(s):
    return (_OWN if own else _PLAIN)[s["op"]](s)


def _own_norm(s):
    import expert_slot_cache_lru_gb300 as m
    kind = {"none": m.MOE_GATE_NONE, "channel": m.MOE_GATE_LINEAR,
            "sigmoid_rows": m.MOE_GATE_SIGMOID}[s["gate"]]
    m.moe_block_norm(s["h"], s["y"], s["post_w"], s["gatev"], s["pre_w"], s["h_out"], s["x_out"],
                     s["rows"], s["hidden"], res_dtype=m.MOE_T_BF16 if s["res"] == "bf16" else m.MOE_T_F32,
                     gate_kind=kind, gate_stride=s["hidden"] if s["gate"] == "sigmoid_rows" else 0,
                     alpha=s["alpha"], w_offset=s["offset"], eps=1e-6)
    return s["h_out"], s["x_out"]


def _own_route(s):
    import expert_slot_cache_lru_gb300 as m
    m.moe_route(s["x"], s["router"], s["biasv"], s["rows"], s["hidden"], s["experts"], s["k"],
                s["logits"], s["ids"], s["w"],
                score=m.MOE_SCORE_SOFTMAX if s["score"] == "softmax" else m.MOE_SCORE_SIGMOID,
                n_groups=s["groups"], topk_groups=s["topk_groups"], group_top=s["group_top"],
                renorm=s["renorm"], scale=s["scale"])
    return s["logits"], s["ids"], s["w"]


def _own_quantize(s):
    import expert_slot_cache_lru_gb300 as m
    fmt = m.MOE_W_NVFP4 if s["fmt"] == "nvfp4" else m.MOE_W_MXFP4
    t = m.MOE_T_BF16 if s["src"] == "bf16" else m.MOE_T_F32
    m.moe_fp4_quantize(fmt, s["src_t"], t, s["rows"], s["cols"], s["glob"], s["codes"], s["scales"])
    m.moe_fp4_dequantize(fmt, s["codes"], s["scales"], s["glob"], s["rows"], s["cols"], s["values"], t)
    return s["values"]


def _own_linear(s):
    import expert_slot_cache_lru_gb300 as m
    fmt = m.MOE_W_NVFP4 if s["fmt"] == "nvfp4" else m.MOE_W_MXFP4
    m.moe_fp4_quantize(fmt, s["x"], m.MOE_T_BF16, s["rows"], s["k"], s["xg"], s["xc"], s["xs"])
    m.moe_fp4_linear(fmt, s["xc"], s["xs"], s["xg"], s["wc"], s["ws"], s["wg"], s["rows"], s["n"],
                     s["k"], s["y"], m.MOE_T_BF16 if s["out"] == "bf16" else m.MOE_T_F32)
    return s["y"]


def _norm_terms(s, t, eps=1e-6):
    """The block norm in the type t: 32 bits for the plain form."""
    z = s["y"].to(t)
    if s["post_w"] is not None:
        z = z * torch.rsqrt(z.square().mean(1, keepdim=True) + eps) * (s["offset"] + s["post_w"].to(t))
    if s["gate"] == "channel":
        z = z * s["gatev"].to(t)
    elif s["gate"] == "sigmoid_rows":
        z = z / (1 + torch.exp(-s["gatev"].to(t)))
    h = s["h"].to(t) + s["alpha"] * z
    x = h * torch.rsqrt(h.square().mean(1, keepdim=True) + eps) * (s["offset"] + s["pre_w"].to(t))
    return h, x


def _plain_norm(s):
    h, x = _norm_terms(s, torch.float32)
    return h.to(s["h"].dtype), x.to(torch.bfloat16)


def _scores(s, z):
    if s["score"] == "softmax":
        e = torch.exp(z - z.max(1, keepdim=True).values)
        return e / e.sum(1, keepdim=True)
    return 1 / (1 + torch.exp(-z))


def _group_scores(s, sc, choice):
    # one best of a group without a bias is ranked by the logits, like the experts
    per = (choice if s["biasv"] is not None or s["group_top"] == 1 else sc).reshape(
        sc.shape[0], s["groups"], -1)
    return per.sort(dim=2, descending=True).values[:, :, :s["group_top"]].sum(2)


def _choice(s, z):
    """Scores, what ranks the experts (the logits where no bias is added) and the eligible ones."""
    sc = _scores(s, z)
    choice = z if s["biasv"] is None else sc + s["biasv"].to(z.dtype)
    eligible = torch.ones_like(z, dtype=torch.bool)
    if s["groups"] > 1:
        order = _group_scores(s, sc, choice).sort(dim=1, descending=True, stable=True).indices
        chosen = torch.zeros(z.shape[0], s["groups"], dtype=torch.bool, device=z.device)
        chosen.scatter_(1, order[:, :s["topk_groups"]], True)
        eligible = chosen.repeat_interleave(z.shape[1] // s["groups"], 1)
    return sc, choice, eligible


def _plain_route(s):
    z = s["x"].float() @ s["router"].float().T
    sc, choice, eligible = _choice(s, z)
    order = choice.masked_fill(~eligible, -math.inf).sort(dim=1, descending=True, stable=True).indices
    ids = order[:, :s["k"]]
    w = sc.gather(1, ids)
    if s["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return z, ids.to(torch.int32), w * s["scale"]


def _nearest_code(a):
    """Index into E2M1 of the nearest value of a >= 0, ties to the even index."""
    return ((a > 0.25).to(torch.int8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
            + (a >= 3.5) + (a > 5.0)).int()


def _quantize(x, glob, fmt):
    """(code values [B][K], block scales [B][K / block] as fp32) of x in 32 bits."""
    blk = 16 if fmt == "nvfp4" else 32
    b = x.reshape(x.shape[0], -1, blk)
    amax = b.abs().amax(2)
    if fmt == "nvfp4":
        scale = torch.clamp(amax / (6.0 * glob), max=448.0).to(torch.float8_e4m3fn).float()
        step = scale * glob
    else:
        scale = torch.exp2(torch.clamp(torch.frexp(amax).exponent - 3.0, -127.0, 127.0))
        step = scale
    div = torch.where(step > 0, step, torch.ones_like(step)).unsqueeze(2)
    q = torch.tensor(E2M1, device=x.device)[_nearest_code((b / div).abs())]
    q = torch.where((step > 0).unsqueeze(2), torch.copysign(q, b), torch.zeros_like(q))
    return q, scale.unsqueeze(2)


def _plain_quantize(s):
    q, sc = _quantize(s["src_t"].float(), s["glob"], s["fmt"])
    v = q * sc if s["glob"] is None else q * sc * s["glob"]
    return v.reshape(s["rows"], s["cols"]).to(s["values"].dtype)


def _weights(s, t=torch.float32):
    """The weights [N][K] without their global scale; products of 4 and 8 bits are exact."""
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=DEV, dtype=t)
    q = torch.stack((table[(s["wc"] & 15).int()], table[(s["wc"] >> 4).int()]), 2)
    if s["fmt"] == "nvfp4":
        sc = s["ws"].view(torch.float8_e4m3fn).to(t)
    else:
        sc = torch.exp2(s["ws"].to(t) - 127)
    return (q.reshape(s["n"], sc.shape[1], -1) * sc.unsqueeze(2)).reshape(s["n"], s["k"])


def _plain_linear(s):
    q, sc = _quantize(s["x"].float(), s["xg"], s["fmt"])
    y = (q * sc).reshape(s["rows"], s["k"]) @ _weights(s).T
    if s["xg"] is not None:
        y = y * (s["xg"] * s["wg"])
    return y.to(s["y"].dtype)


_OWN = {"norm": _own_norm, "route": _own_route, "quantize": _own_quantize, "linear": _own_linear}
_PLAIN = {"norm": _plain_norm, "route": _plain_route, "quantize": _plain_quantize,
          "linear": _plain_linear}


# ------------------------------------------------------------------- the floor

def work(c):
    """Bytes read and written once and operations of one pass."""
    if c["op"] == "norm":
        n, r = c["rows"] * c["hidden"], 2 if c["res"] == "bf16" else 4
        gate = {"none": 0, "channel": 2 * c["hidden"], "sigmoid_rows": 2 * n}[c["gate"]]
        return {"bytes": n * (2 * r + 4) + gate + 2 * c["hidden"] * (1 + c["post"]),
                "flops": 12 * n}
    if c["op"] == "route":
        n = c["rows"] * c["experts"]
        return {"bytes": 2 * c["hidden"] * (c["rows"] + c["experts"]) + 4 * n + 8 * c["rows"] * c["k"],
                "flops": 2 * n * c["hidden"]}
    if c["op"] == "quantize":
        # source in, codes and scales out and in again, values out
        n, r = c["rows"] * c["cols"], 2 if c["src"] == "bf16" else 4
        return {"bytes": 2 * n * r + 2 * (n // 2 + n // (16 if c["fmt"] == "nvfp4" else 32)),
                "flops": 6 * n}
    m, k, n = c["rows"], c["k"], c["n"]
    blk = 16 if c["fmt"] == "nvfp4" else 32
    return {"bytes": 2 * m * k + n * (k // 2 + k // blk) + m * n * (2 if c["out"] == "bf16" else 4),
            "flops": 2 * m * k * n}


# ------------------------------------------------------------------- 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s)
    if case["op"] == "route":
        return _exact_route(s)
    if case["op"] == "quantize":
        q, sc = _exact_quantize(s["src_t"].double(), s["glob"], s["fmt"])
        v = (q * sc.unsqueeze(2)).reshape(s["rows"], s["cols"])
        return v if s["glob"] is None else v.mul_(s["glob"].double())
    q, sc = _exact_quantize(s["x"].double(), s["xg"], s["fmt"])
    a = (q * sc.unsqueeze(2)).reshape(s["rows"], s["k"])
    y = a @ _exact_weights(s).T
    return y if s["xg"] is None else y * (s["xg"].double() * s["wg"].double())


def _exact_norm(s):
    d = torch.float64
    H = s["hidden"]
    y, h = s["y"].to(d), s["h"].to(d)
    if s["post_w"] is not None:
        rms = (torch.einsum("bh,bh->b", y, y) / H + 1e-6).sqrt()
        y = torch.einsum("bh,h,b->bh", y, s["post_w"].to(d) + s["offset"], 1 / rms)
    if s["gatev"] is not None:
        gate = s["gatev"].to(d)
        y = y * (torch.special.expit(gate) if s["gate"] == "sigmoid_rows" else gate)
    h = torch.add(h, y, alpha=s["alpha"])
    rms = (torch.einsum("bh,bh->b", h, h) / H + 1e-6).sqrt()
    return h, torch.einsum("bh,h,b->bh", h, s["pre_w"].to(d) + s["offset"], 1 / rms)


def _exact_route(s):
    z = torch.einsum("bh,eh->be", s["x"].double(), s["router"].double())
    p = torch.softmax(z, 1) if s["score"] == "softmax" else torch.special.expit(z)
    rank = p if s["biasv"] is None else p + s["biasv"].double()
    B, E, G = z.shape[0], z.shape[1], s["groups"]
    if G > 1:
        best = rank.view(B, G, E // G).topk(s["group_top"], 2).values.sum(2)
        keep = best >= best.topk(s["topk_groups"], 1).values[:, -1:]
        rank = torch.where(keep.unsqueeze(2), rank.view(B, G, E // G), -math.inf).view(B, E)
    ids = rank.topk(s["k"], 1).indices
    w = p.gather(1, ids)
    if s["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return z, None, w * s["scale"]


def _to_grid(v, grid):
    """Nearest value of a sorted grid of nonnegative values, ties to the even index."""
    mid = (grid[1:] + grid[:-1]) / 2
    i = torch.bucketize(v, mid)                      # v in (mid[i-1], mid[i]]
    tie = (i < mid.numel()) & (v == mid[i.clamp(max=mid.numel() - 1)])
    return grid[i + (tie & (i % 2 == 1)).long()]


def _exact_quantize(x, glob, fmt):
    blk = 16 if fmt == "nvfp4" else 32
    g = torch.ones(1, dtype=torch.float64, device=DEV) if glob is None else glob.double()
    b = x.view(x.shape[0], -1, blk)
    amax = b.abs().max(2).values
    if fmt == "nvfp4":
        e4m3 = [m * 2.0 ** -9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16)
                                                    for m in range(8) if (e, m) != (15, 7)]
        sc = _to_grid(amax / (6 * g), torch.tensor(e4m3, dtype=torch.float64, device=DEV))
    else:
        # the logarithm of a power of two may come out a little low; 1e-9 is far below the inputs' steps
        sc = torch.exp2(torch.floor(torch.log2(amax) + 1e-9).clamp(min=-125.0) - 2)
    step = (sc * g).unsqueeze(2)
    q = _to_grid((b / step).abs().nan_to_num(0.0), torch.tensor(E2M1, dtype=torch.float64, device=DEV))
    return torch.where(step > 0, torch.sign(b) * q, 0.0), sc


def _exact_weights(s):
    c = torch.empty(s["n"], s["k"], dtype=torch.float64, device=DEV)
    for half, bits in ((0, s["wc"] % 16), (1, s["wc"] // 16)):
        e, m = (bits % 8) // 2, (bits % 2).double()
        v = torch.where(e == 0, m / 2, (1 + m / 2) * torch.exp2(e.double() - 1))
        c[:, half::2] = torch.where(bits >= 8, -v, v)
    if s["fmt"] == "nvfp4":
        e, m = s["ws"] // 8, (s["ws"] % 8).double()
        sc = torch.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * torch.exp2(e.double() - 7))
    else:
        sc = torch.exp2(s["ws"].double() - 127)
    return c.view(s["n"], sc.shape[1], -1).mul_(sc.unsqueeze(2)).view(s["n"], s["k"])

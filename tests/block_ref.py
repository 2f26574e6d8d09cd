"""The operators around the experts in 64 bits (numpy), for the tests: formulas
as in include/moe_cache.h, written without the library's code."""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([m * 2.0 ** -9 for m in range(8)] +
                [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)][:-1])


def block_norm(h, y=None, post_w=None, gate=None, gate_kind="none", alpha=1.0, pre_w=None,
               offset=0.0, eps=1e-6):
    """(h', x', size of the terms h' is summed from)."""
    size = np.abs(h)
    if y is not None:
        z = y
        if post_w is not None:
            z = z / np.sqrt((z * z).mean(1, keepdims=True) + eps) * (offset + post_w)
        if gate_kind == "linear":
            z = z * gate
        elif gate_kind == "sigmoid":
            z = z / (1 + np.exp(-gate))
        size = size + np.abs(alpha * z)
        h = h + alpha * z
    x = None
    if pre_w is not None:
        x = h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * (offset + pre_w)
    return h, x, size


def choice(z, score, bias):
    """Scores and choices of logits z [rows][E]; NaN marks a masked expert's choice."""
    masked = np.isnan(z) | (z == -np.inf)
    zz = np.where(masked, -np.inf, z)
    if score == "softmax":
        mx = zz.max(1, keepdims=True)
        with np.errstate(invalid="ignore"):
            e = np.where(mx == np.inf, (zz == np.inf).astype(float),
                         np.where(masked, 0.0, np.exp(zz - np.where(np.isfinite(mx), mx, 0.0))))
        tot = e.sum(1, keepdims=True)
        s = np.divide(e, tot, out=np.zeros_like(e), where=tot > 0)
    else:
        s = np.where(masked, 0.0, 1 / (1 + np.exp(-np.where(masked, 0.0, zz))))
    c = z if bias is None else s + bias
    c = np.where(masked | np.isnan(c) | (c == -np.inf), np.nan, c)
    return s, c


def route(z, k, score="softmax", bias=None, groups=1, topk_groups=1, group_top=1, renorm=True,
          scale=1.0):
    """(ids [rows][k], weights, smallest gap between two different ranked values)."""
    z = np.asarray(z, dtype=np.float64)
    s, c = choice(z, score, bias)
    B, E = z.shape
    ids = np.full((B, k), -1, np.int64)
    w = np.zeros((B, k))
    gap = np.inf
    for b in range(B):
        ok = ~np.isnan(c[b])
        if groups > 1:
            gsc = []
            for g in range(groups):
                part = slice(g * (E // groups), (g + 1) * (E // groups))
                by = s[b] if (bias is None and group_top == 2) else c[b]
                v = np.sort(by[part][~np.isnan(c[b][part])])[::-1][:group_top]
                gsc.append(v.sum() if v.size else np.nan)
            order = [g for g in sorted(range(groups), key=lambda g: (-gsc[g] if gsc[g] == gsc[g] else np.inf, g))
                     if gsc[g] == gsc[g]]
            r = np.sort(np.array(gsc)[order])
            d = np.diff(r)
            gap = min([gap, *d[d > 0]])
            keep = set(order[:topk_groups])
            ok &= np.array([e // (E // groups) in keep for e in range(E)])
        cand = np.nonzero(ok)[0]
        pick = cand[np.argsort(-c[b][cand], kind="stable")]
        with np.errstate(invalid="ignore"):
            d = -np.diff(c[b][pick][:k + 1])
        gap = min([gap, *d[d > 0]])
        pick = pick[:k]
        ids[b, :pick.size] = pick
        w[b, :pick.size] = s[b][pick]
    if renorm:
        t = w.sum(1, keepdims=True)
        w = np.divide(w, t, out=np.zeros_like(w), where=t > 0)
    return ids, w * scale, gap


def nearest(v, grid):
    """Index of the nearest value of a sorted grid, ties to the even index, saturating."""
    v = np.asarray(v, np.float64)
    i = np.clip(np.searchsorted(grid, v), 1, len(grid) - 1)
    lo, hi = grid[i - 1], grid[i]
    up = (v - lo > hi - v) | ((v - lo == hi - v) & (i % 2 == 0))
    return np.where(up, i, i - 1)


def quantize(x, nv, g=None):
    """(codes [rows][cols/2], scales) in the fp32 steps the header states (x float32)."""
    x = np.asarray(x, np.float32)
    B, K = x.shape
    blk = 16 if nv else 32
    b = x.reshape(B, K // blk, blk)
    nan = np.isnan(b).any(2)
    amax = np.nan_to_num(np.abs(b), nan=0.0, posinf=np.inf).max(2).astype(np.float32)
    with np.errstate(all="ignore"):
        if nv:
            gl = np.float32(1.0 if g is None else g)
            t = np.minimum(amax / (np.float32(6) * gl), np.float32(448))
            sc = nearest(t, E4M3).astype(np.uint8)
            step = (E4M3[sc].astype(np.float32) * gl).astype(np.float32)
        else:
            ex = np.where(np.isinf(amax), 128, np.frexp(amax)[1] - 1)
            ex = np.where(amax == 0, -200, ex) - 2
            sc = np.clip(ex + 127, 0, 254).astype(np.uint8)
            step = np.ldexp(np.float64(1), sc.astype(np.int64) - 127).astype(np.float32)
        q = (b / step[..., None]).astype(np.float32)
        idx = nearest(np.abs(q).clip(max=1e6), E2M1).astype(np.uint8)
    code = np.where((step > 0)[..., None], idx | (np.signbit(b).astype(np.uint8) << 3), 0)
    code = np.where(nan[..., None], 0, code).reshape(B, K).astype(np.uint8)
    sc = np.where(nan, 0x7F if nv else 0xFF, sc).astype(np.uint8)
    return code[:, ::2] | (code[:, 1::2] << 4), sc


def decode(codes, scales, nv, g=None):
    """Values [rows][cols] of code and scale banks, in 64 bits."""
    t = np.concatenate([E2M1, -E2M1])
    B = codes.shape[0]
    q = np.stack([t[codes & 15], t[codes >> 4]], 2).reshape(B, scales.shape[1], -1)
    if nv:
        e = np.concatenate([E4M3, [np.nan]])
        sc = np.concatenate([e, -e])[scales]
    else:
        sc = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    v = (q * sc[..., None]).reshape(B, -1)
    return v if g is None else v * np.float64(np.float32(g))

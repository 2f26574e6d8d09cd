"""The bf16 products, the order of routes and the combine in 64 bits, with bounds of
what fp32 operations may be off by."""
import math

import numpy as np
import torch

U = 2.0 ** -24
ACTS = ("none", "silu", "gelu", "gelu_tanh", "relu")


def act_id(m, name):
    return getattr(m, "MOE_ACT_" + name.upper())


def half_step(dtype):
    return 2.0 ** -8 if dtype == torch.bfloat16 else U


def act(z, kind):
    """(act(z), bound of its evaluation's error in fp32) in 64 bits."""
    if kind == "silu":
        y, arg = z * torch.special.expit(z), z.abs()
    elif kind == "gelu":
        y, arg = z * 0.5 * torch.special.erfc(-z * math.sqrt(0.5)), torch.zeros_like(z)  # ndtr cancels below -8
    elif kind == "gelu_tanh":
        u2 = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
        y, arg = z * torch.special.expit(u2), u2.abs()
    elif kind == "relu":
        y = torch.where(z < 0, torch.zeros_like(z), z)
        return y, torch.zeros_like(z)
    else:
        return z, torch.zeros_like(z)
    # e^-arg: arg is off by a few roundings of its size, the exponential by 2 ulp, normcdff by 5 ulp;
    # quotient and products by 4.  Below fp32's smallest normal number: that number.
    return y, (16 + 8 * arg.clamp(max=200)) * U * y.abs() + 2.0 ** -126 * (1 + z.abs())


def product(x, w, bias, kind, gated, chain):
    """(y, bound) of act(x w^T + bias) (or gated), `chain` the roundings of U that a sum of absolute
    size 1 may be off by."""
    d = torch.float64
    x, w = x.to(d), w.to(d)
    z, size = x @ w.T, x.abs() @ w.abs().T
    if bias is not None:
        z, size = z + bias.to(d), size + bias.to(d).abs()
    dz = (chain + 2) * U * size
    if not gated:
        y, e = act(z, kind)
        return y, e + 1.13 * dz          # no activation is steeper than 1.13
    n = z.shape[1] // 2
    a, e = act(z[:, :n], kind)
    e = e + 1.13 * dz[:, :n]
    u, du = z[:, n:], dz[:, n:]
    return a * u, e * (u.abs() + du) + a.abs() * du + U * (a * u).abs()


def check(out, y, dy, dtype, alpha=1.0, res=None):
    want, err = alpha * y, abs(alpha) * dy + 2 * U * (alpha * y).abs()
    if res is not None:
        want, err = want + res.double(), err + 2 * U * res.double().abs()
    err = err + half_step(dtype) * (want.abs() + err) + 2.0 ** -133
    off = (out.double() - want).abs()
    bad = ~(off <= err)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(), float((off / err).nan_to_num(99).max()))


def group(ids, E):
    """(offsets, order, pos) of a flat int array."""
    ids = np.asarray(ids, np.int64).reshape(-1)
    ok = (ids >= 0) & (ids < E)
    routes = np.flatnonzero(ok)
    placed = routes[np.argsort(ids[routes], kind="stable")]
    offsets = np.concatenate(([0], np.cumsum(np.bincount(ids[routes], minlength=E)))).astype(np.int32)
    order = np.full(ids.size, -1, np.int32)
    order[:placed.size] = placed
    pos = np.full(ids.size, -1, np.int32)
    pos[placed] = np.arange(placed.size)
    return offsets, order, pos

"""The bf16 products, the grouping of routes and the combine on the GPU, against
their formulas in 64 bits (linear_ref.py has the bounds)."""
import zlib

import numpy as np
import pytest
import torch

from tests import linear_ref as ref

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def m():
    import expert_slot_cache_lru_gb300 as mod
    return mod


def gen(*key):
    return torch.Generator(device="cuda").manual_seed(zlib.crc32(repr(key).encode()))


def normal(g, *shape, std=1.0, dtype=BF16):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def padded(t, pad=0, off=0, fill=float("nan")):
    """A copy of the rows of t (last dimension) inside a larger buffer of `fill`."""
    rows, cols = t.numel() // t.shape[-1], t.shape[-1]
    big = torch.full((rows * (cols + pad) + off,), fill, dtype=t.dtype, device="cuda")
    v = big[off:].view(*t.shape[:-1], cols + pad)[..., :cols]
    v.copy_(t)
    return v


def chain(K, whole):
    """Roundings of a sum of K products: eight of U for 16 of K in the tensor cores (truncated additions of
    16 products to a sum) or across 32 lanes of dot products; one each in the CUDA-core tiles."""
    return K / 2 + 40 if whole else K + 8


def linear_case(m, B, N, K, *, kind="none", gated=False, bias=False, res=False, alpha=1.0, f32=False, pad=0,
                off=0, alias=False, scale=1.0, bound=None):
    g = gen(B, N, K, kind, gated)
    t = torch.float32 if f32 else BF16
    wide = N * (1 + gated)
    x = padded(normal(g, B, K, std=scale), pad, off)
    w = padded(normal(g, wide, K, std=K ** -0.5), pad, off)
    b = normal(g, wide, std=0.5) if bias else None
    r = padded(normal(g, B, N, std=3.0, dtype=t), pad, off) if res else None
    kept = r.clone() if res else None
    out = r if alias else padded(torch.zeros(B, N, dtype=t, device="cuda"), pad, off, fill=-7.0)
    whole = out.storage_offset(), out.untyped_storage().nbytes()
    st = torch.zeros(1, dtype=torch.int64, device="cuda")
    m.moe_linear(x, w, b, r, out, B, N, K, act=ref.act_id(m, kind), gated=gated, alpha=alpha,
                 dtype=m.MOE_T_F32 if f32 else m.MOE_T_BF16, x_stride=K + pad, w_stride=K + pad,
                 res_stride=N + pad, out_stride=N + pad, d_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0 and whole[0] == off
    ok = K % 8 == 0 and pad % 8 == 0 and off % 8 == 0
    y, dy = ref.product(x, w, b, kind, gated, bound or chain(K, ok))
    ref.check(out, y, dy, t, alpha, kept)
    if pad and not alias:  # nothing beside the rows is written
        flat = out.as_strided((B, N + pad), (N + pad, 1), off)
        assert (flat[:, N:] == -7.0).all()
    return out


# rows and widths around every tile's edges
@pytest.mark.parametrize("B", [1, 2, 3, 4, 5, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 200, 255,
                               256, 257, 300, 512, 513])
@pytest.mark.parametrize("N,K", [(128, 64), (200, 136), (1, 8), (513, 320)])
def test_linear_rows(m, B, N, K):
    linear_case(m, B, N, K, bias=True)


@pytest.mark.parametrize("N", [1, 2, 7, 16, 31, 32, 33, 64, 100, 127, 128, 129, 255, 256, 257, 511, 1000, 2048])
@pytest.mark.parametrize("B", [1, 6, 40, 300])
def test_linear_widths(m, B, N):
    linear_case(m, B, N, 192, res=True, alpha=0.5)


@pytest.mark.parametrize("K", [1, 2, 7, 8, 9, 16, 24, 63, 64, 65, 72, 120, 128, 136, 255, 256, 264, 1000, 1024, 2040,
                               2048, 2056, 4104, 8192])
@pytest.mark.parametrize("B", [1, 3, 20, 150])
def test_linear_depths(m, B, K):
    linear_case(m, B, 144, K, bias=True, f32=True)


@pytest.mark.parametrize("kind", ref.ACTS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("B,K", [(1, 512), (4, 200), (37, 512), (260, 264), (33, 77)])
def test_linear_forms(m, kind, gated, f32, B, K):
    linear_case(m, B, 208, K, kind=kind, gated=gated, bias=True, res=True, alpha=0.22, f32=f32, scale=2.0)


@pytest.mark.parametrize("kw", [dict(pad=8), dict(pad=24, off=8), dict(pad=1), dict(off=1), dict(pad=3, off=5),
                                dict(alias=True, res=True), dict(alias=True, res=True, pad=8, f32=True),
                                dict(alias=True, res=True, pad=1)])
@pytest.mark.parametrize("B,N,K,gated", [(1, 300, 512, False), (3, 64, 256, True), (50, 304, 512, True),
                                         (300, 515, 200, False), (270, 96, 328, True)])
def test_linear_layouts(m, kw, B, N, K, gated):
    linear_case(m, B, N, K, gated=gated, kind="silu", bias=True, **kw)


@pytest.mark.parametrize("N", [1, 8, 15, 17, 40, 130])
@pytest.mark.parametrize("B", [2, 30, 300])
def test_linear_gated_odd_widths(m, B, N):
    linear_case(m, B, N, 256, gated=True, kind="gelu", bias=True)


@pytest.mark.parametrize("B,N,K,gated", [(1, 4096, 4096, False), (4, 3000, 2048, False), (16, 2048, 2048, False),
                                         (64, 1024, 4096, True), (600, 768, 2048, True), (1333, 1001, 2072, False),
                                         (2000, 4096, 1024, False), (700, 2048, 512, True), (5000, 640, 768, False)])
@pytest.mark.parametrize("f32", [False, True])
def test_linear_larger(m, B, N, K, gated, f32):
    linear_case(m, B, N, K, gated=gated, kind="gelu_tanh", bias=True, res=True, f32=f32)


def test_linear_zero_rows_leave_everything(m):
    out = torch.full((4, 8), 3.0, dtype=BF16, device="cuda")
    m.moe_linear(out, out, None, None, None, 0, 8, 8)
    torch.cuda.synchronize()
    assert (out == 3).all()


@pytest.mark.parametrize("B", [1, 3, 40, 300])
@pytest.mark.parametrize("kind", ref.ACTS)
def test_linear_nan_and_infinity_stay_in_their_rows(m, B, kind):
    N, K = 160, 256
    g = gen(B, 1)
    x, w = normal(g, B, K), normal(g, N, K)
    bad = w.clone()
    bad[3, 5], bad[130, 7] = float("nan"), float("inf")
    a, b = (torch.empty(B, N, dtype=BF16, device="cuda") for _ in range(2))
    m.moe_linear(x, w, None, None, a, B, N, K, act=ref.act_id(m, kind))
    m.moe_linear(x, bad, None, None, b, B, N, K, act=ref.act_id(m, kind))
    assert b[:, 3].isnan().all()
    up = x[:, 7].float() > 0
    assert (b[up, 130] == float("inf")).all()
    down = b[x[:, 7].float() < 0, 130]
    if kind == "relu":
        assert (down == 0).all()
    elif kind == "none":
        assert (down == float("-inf")).all()
    else:
        assert down.isnan().all()
    keep = [i for i in range(N) if i not in (3, 130)]
    assert torch.equal(a[:, keep], b[:, keep])
    x[0, 0] = float("nan")
    m.moe_linear(x, w, None, None, b, B, N, K, act=ref.act_id(m, kind))
    assert b[0].isnan().all() and torch.equal(a[1:], b[1:])


@pytest.mark.parametrize("kind", ["silu", "gelu", "gelu_tanh"])
def test_activations_over_their_range(m, kind):
    """z passes through exactly (an identity as weights): every size from the tails to the largest."""
    K = 64
    z = torch.cat([torch.linspace(-110, 30, 3000), torch.linspace(-3, 3, 2000), torch.tensor([0.0, -0.0, 1e30, -1e30])])
    x = torch.zeros(z.numel(), K, dtype=BF16, device="cuda")
    x[:, 5] = z.to(BF16).cuda()
    w = torch.eye(K, dtype=BF16, device="cuda")
    for rows in (1, 3, 5004):
        out = torch.empty(rows, K, device="cuda")
        m.moe_linear(x[:rows], w, None, None, out, rows, K, K, act=ref.act_id(m, kind), dtype=m.MOE_T_F32)
        y, e = ref.act(x[:rows, 5].double(), kind)
        e = e + ref.U * y.abs()
        assert ((out[:, 5].double() - y).abs() <= e).all()


def test_linear_equal_inputs_give_equal_bits(m):
    for B, N, K in ((1, 512, 1024), (30, 512, 4096), (600, 1024, 2048)):
        g = gen(B, N, K)
        x, w = normal(g, B, K), normal(g, N, K)
        outs = []
        for _ in range(4):
            o = torch.empty(B, N, device="cuda")
            m.moe_linear(x, w, None, None, o, B, N, K, dtype=m.MOE_T_F32)
            outs.append(o)
        assert all(torch.equal(outs[0], o) for o in outs[1:])


# ------------------------------------------------------------------ order of routes

def group_case(m, ids, E, in_place=False):
    ids = np.asarray(ids, np.int32)
    R = ids.size
    t = torch.from_numpy(ids.copy()).cuda()
    offsets = torch.full((E + 1,), -9, dtype=torch.int32, device="cuda")
    order = torch.full((R + 3,), -9, dtype=torch.int32, device="cuda")
    pos = t if in_place else torch.full((R + 3,), -9, dtype=torch.int32, device="cuda")
    m.moe_group_routes(t, R, E, offsets, order, pos)
    want = ref.group(ids, E)
    assert np.array_equal(offsets.cpu().numpy(), want[0])
    assert np.array_equal(order.cpu().numpy()[:R], want[1]) and (order[R:] == -9).all()
    assert np.array_equal(pos.cpu().numpy()[:R], want[2]) and (in_place or (pos[R:] == -9).all())


@pytest.mark.parametrize("R", [0, 1, 2, 8, 31, 32, 33, 255, 256, 257, 1000, 1024, 1025, 4097, 8191, 65536, 100001])
@pytest.mark.parametrize("E", [1, 2, 8, 60, 256, 1000, 1024, 1025])
def test_group_routes(m, R, E):
    r = np.random.default_rng([R, E])
    ids = r.integers(-1, E + 1, R)
    ids[r.random(R) < 0.3] = r.integers(0, E)   # one crowded expert
    group_case(m, ids, E)


@pytest.mark.parametrize("R,E", [(5, 16384), (3000, 16384), (70000, 16384), (70000, 3164), (600000, 5), (2000000, 300)])
def test_group_routes_large(m, R, E):
    r = np.random.default_rng([R, E])
    group_case(m, r.integers(-2, E + 2, R), E)


@pytest.mark.parametrize("ids", [[], [-1], [0] * 40, [-1] * 2000, [7] * 5000, [2 ** 31 - 1, -2 ** 31, 0, 3]])
def test_group_routes_extremes(m, ids):
    group_case(m, ids, 8)


@pytest.mark.parametrize("R", [7, 900, 20000])
def test_group_routes_in_place_and_without_order(m, R):
    r = np.random.default_rng(R)
    ids = r.integers(-1, 50, R).astype(np.int32)
    group_case(m, ids, 50, in_place=True)
    t = torch.from_numpy(ids).cuda()
    offsets = torch.empty(51, dtype=torch.int32, device="cuda")
    pos = torch.empty_like(t)
    m.moe_group_routes(t, R, 50, offsets)
    m.moe_group_routes(t, R, 50, offsets, None, pos)
    want = ref.group(ids, 50)
    assert np.array_equal(offsets.cpu().numpy(), want[0]) and np.array_equal(pos.cpu().numpy(), want[2])


# ------------------------------------------------------------------ products of groups

def grouped_case(m, counts, N, K, *, kind="none", gated=False, bias=False, f32=False, gather=True, top=2, gap=0,
                 pad=0, off=0, spare=3, bad=0):
    """counts: rows of each group.  spare: rows of out behind the last group; bad: places whose order
    names no row."""
    g = gen(len(counts), N, K, kind, gated, gather)
    E, placed, wide = len(counts), int(sum(counts)), N * (1 + gated)
    rows = placed + spare
    t = torch.float32 if f32 else BF16
    offsets = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device="cuda")
    x_rows = max(1, (rows + top - 1) // top) if gather else rows
    x = padded(normal(g, x_rows, K), pad, off)
    order = None
    if gather:
        order = torch.full((rows,), -1, dtype=torch.int32, device="cuda")
        order[:placed] = torch.randperm(x_rows * top, generator=g, device="cuda")[:placed].int()
        if bad and placed:
            at = torch.randperm(placed, generator=g, device="cuda")[:bad]
            order[at] = torch.tensor([-1, x_rows * top, -2 ** 31, 2 ** 31 - 1], dtype=torch.int32,
                                     device="cuda")[torch.arange(at.numel(), device="cuda") % 4]
    ws = K + pad
    big = torch.full((E * (wide * ws + gap) + off,), float("nan"), dtype=BF16, device="cuda")
    w = big[off:].as_strided((E, wide, K), (wide * ws + gap, ws, 1), off)
    w.copy_(normal(g, E, wide, K, std=K ** -0.5))
    for e, c in enumerate(counts):
        if c == 0:
            w[e] = float("nan")      # may be unset
    b = normal(g, E, wide, std=0.5) if bias else None
    out = padded(torch.full((rows, N), -7.0, dtype=t, device="cuda"), pad, off, fill=-7.0)
    st = torch.zeros(1, dtype=torch.int64, device="cuda")
    m.moe_grouped_linear(x, x_rows, order, top, offsets, E, w, b, out, rows, N, K, act=ref.act_id(m, kind),
                         gated=gated, dtype=m.MOE_T_F32 if f32 else m.MOE_T_BF16, x_stride=K + pad, w_stride=ws,
                         w_group_stride=wide * ws + gap, out_stride=N + pad, d_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    ok = K % 8 == 0 and pad % 8 == 0 and off % 8 == 0 and gap % 8 == 0
    at = 0
    for e, c in enumerate(counts):
        if c:
            src = torch.arange(at, at + c, device="cuda")
            o = out[at:at + c]
            if gather:
                src = order[at:at + c].long()
                good = (src >= 0) & (src < x_rows * top)
                assert (o[~good] == -7).all()
                src, o = src[good] // top, o[good]
            y, dy = ref.product(x[src], w[e], b[e] if bias else None, kind, gated, chain(K, ok))
            ref.check(o, y, dy, t)
        at += c
    assert (out[placed:] == -7).all()
    if pad:
        assert (out.as_strided((rows, N + pad), (N + pad, 1), off)[:, N:] == -7).all()


COUNTS = {
    "one": [1], "none": [0, 0, 0], "few": [0, 3, 1, 0, 2], "single": [0] * 100 + [1] + [0] * 155,
    "token": [1 if e % 32 == 5 else 0 for e in range(256)],
    "edges": [15, 16, 17, 31, 32, 33, 0, 63, 64, 65, 127, 128, 129, 255, 256, 257, 0],
    "crowded": [700, 0, 0, 3], "last": [0] * 300 + [5], "sparse": [e % 3 for e in range(200)],
    "many": [(e * 7) % 5 for e in range(1500)],
}


@pytest.mark.parametrize("name", COUNTS)
@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("N,K,gated", [(64, 128, True), (144, 72, False), (300, 264, False)])
def test_grouped_counts(m, name, gather, N, K, gated):
    grouped_case(m, COUNTS[name], N, K, gather=gather, gated=gated, kind="silu", bias=True)


@pytest.mark.parametrize("kind", ref.ACTS)
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("f32", [False, True])
def test_grouped_forms(m, kind, gated, f32):
    for counts in ([2, 0, 1, 4], [40, 0, 1, 130, 5]):
        grouped_case(m, counts, 176, 200, kind=kind, gated=gated, bias=True, f32=f32)


@pytest.mark.parametrize("kw", [dict(pad=8), dict(pad=8, off=8, gap=16), dict(gap=1), dict(pad=1), dict(off=1),
                                dict(gap=128, gather=False), dict(top=1), dict(top=8), dict(bad=3), dict(bad=40),
                                dict(spare=0), dict(spare=500), dict(gather=False, pad=8), dict(bad=2, pad=3)])
@pytest.mark.parametrize("counts", [[1, 0, 2, 1], [50, 3, 0, 200], [270]])
@pytest.mark.parametrize("N,K,gated", [(96, 256, True), (130, 136, False)])
def test_grouped_layouts(m, kw, counts, N, K, gated):
    grouped_case(m, counts, N, K, gated=gated, kind="gelu", bias=True, **kw)


@pytest.mark.parametrize("N,K,gated", [(512, 2048, True), (2048, 512, False), (768, 1024, True), (1000, 1032, False)])
@pytest.mark.parametrize("name", ["token", "edges", "sparse"])
def test_grouped_larger(m, name, N, K, gated):
    grouped_case(m, COUNTS[name], N, K, gated=gated, kind="silu")


def test_grouped_offsets_out_of_order_stay_inside(m):
    """Offsets no grouping writes: rows outside [0, n_rows) are never touched."""
    g = gen(5)
    N, K, rows = 64, 64, 40
    x, w = normal(g, rows, K), normal(g, 4, N, K)
    big = torch.full((rows + 20, N), -7.0, dtype=BF16, device="cuda")
    out = big[10:10 + rows]
    for offs in ([-5, 10, 5, 30, 900], [50, 60, 70, 80, 90], [0, 0, 0, 0, 2 ** 31 - 1], [-2 ** 31, -3, -2, -1, 0]):
        o = torch.tensor(offs, dtype=torch.int32, device="cuda")
        m.moe_grouped_linear(x, rows, None, 1, o, 4, w, None, out, rows, N, K)
        torch.cuda.synchronize()
        assert (big[:10] == -7).all() and (big[10 + rows:] == -7).all()


# ------------------------------------------------------------------ the combine

def combine_case(m, B, k, H, *, y32=False, f32=False, add=True, pad=0, off=0, alias=False, drop=0.2):
    g = gen(B, k, H, y32, f32)
    t, ty = torch.float32 if f32 else BF16, torch.float32 if y32 else BF16
    Y = max(1, B * k - 3)
    y = padded(normal(g, Y, H, dtype=ty), pad, off)
    pos = torch.randint(0, Y, (B, k), generator=g, device="cuda").int()
    gone = torch.rand(B, k, generator=g, device="cuda") < drop
    pos[gone] = torch.tensor([-1, Y, -2 ** 31, 2 ** 31 - 1], dtype=torch.int32, device="cuda")[
        torch.arange(int(gone.sum()), device="cuda") % 4]
    w = torch.randn(B, k, generator=g, device="cuda")
    w[gone] = float("nan")
    a = padded(normal(g, B, H, std=2.0, dtype=t), pad, off) if add else None
    out = a if alias else padded(torch.zeros(B, H, dtype=t, device="cuda"), pad, off, fill=-7.0)
    want = a.double().clone() if add else torch.zeros(B, H, dtype=torch.float64, device="cuda")
    size = want.abs()
    for j in range(k):
        term = y[pos[:, j].clamp(0, Y - 1).long()].double() * w[:, j:j + 1].double()
        term[gone[:, j]] = 0
        want, size = want + term, size + term.abs()
    m.moe_combine(y, Y, pos, w, a, out, B, k, H, y_dtype=m.MOE_T_F32 if y32 else m.MOE_T_BF16,
                  dtype=m.MOE_T_F32 if f32 else m.MOE_T_BF16, y_stride=H + pad, add_stride=H + pad, out_stride=H + pad)
    torch.cuda.synchronize()
    err = (k + 1) * ref.U * size + ref.half_step(t) * want.abs() * 1.01 + 2.0 ** -133
    assert ((out.double() - want).abs() <= err).all()
    if pad and not alias:
        assert (out.as_strided((B, H + pad), (H + pad, 1), off)[:, H:] == -7).all()


@pytest.mark.parametrize("H", [1, 7, 8, 24, 100, 1024, 2048, 4095])
@pytest.mark.parametrize("B,k", [(1, 1), (1, 8), (3, 2), (100, 6), (17, 9), (5, 40)])
@pytest.mark.parametrize("y32,f32", [(False, False), (False, True), (True, True)])
def test_combine(m, B, k, H, y32, f32):
    combine_case(m, B, k, H, y32=y32, f32=f32)


@pytest.mark.parametrize("kw", [dict(add=False), dict(alias=True), dict(pad=8), dict(pad=8, off=8, alias=True),
                                dict(pad=1), dict(off=1), dict(pad=3, off=1, f32=True), dict(drop=1.0),
                                dict(drop=1.0, add=False), dict(drop=0.0, y32=True, f32=True, pad=4)])
@pytest.mark.parametrize("B,k,H", [(1, 8, 2048), (50, 2, 264), (700, 8, 512)])
def test_combine_layouts(m, kw, B, k, H):
    combine_case(m, B, k, H, **kw)


# ------------------------------------------------------------------ together

@pytest.mark.parametrize("B,k,E,H,I", [(1, 8, 64, 512, 256), (5, 2, 16, 256, 96), (150, 4, 32, 512, 128),
                                       (700, 8, 20, 256, 64)])
@pytest.mark.parametrize("captured", [False, True])
def test_a_layer_of_resident_experts(m, B, k, E, H, I, captured):  # noqa: E741
    """Router, order, gate and up, down, combine with a dense expert beside them, over bf16 blobs of a
    slot pool; eager and replayed."""
    g = gen(B, k, E)
    blob, dev = 3 * H * I, dict(device="cuda")
    stride = (2 * blob + 255) // 256 * 128 + 128      # elements; slots with a gap between them
    pool = torch.full((E, stride), float("nan"), dtype=BF16, **dev)
    pool[:, :blob] = normal(g, E, blob, std=H ** -0.5)
    router, dense = normal(g, E, H, std=H ** -0.5), normal(g, 2 * I, H, std=H ** -0.5)
    down = normal(g, H, I, std=I ** -0.5)
    x = torch.empty(B, H, dtype=BF16, **dev)
    z, w = torch.empty(B, E, **dev), torch.empty(B, k, **dev)
    ids = torch.empty(B, k, dtype=torch.int32, **dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, **dev)
    order, pos = (torch.empty(B * k, dtype=torch.int32, **dev) for _ in range(2))
    h, y = torch.zeros(B * k, I, dtype=BF16, **dev), torch.zeros(B * k, H, dtype=BF16, **dev)
    hd, yd, out = (torch.empty(B, n, dtype=BF16, **dev) for n in (I, H, H))

    def step():
        m.moe_route(x, router, None, B, H, E, k, z, ids, w)
        m.moe_group_routes(ids, B * k, E, offsets, order, pos)
        m.moe_grouped_linear(x, B, order, k, offsets, E, pool, None, h, B * k, I, H, act=m.MOE_ACT_SILU, gated=True,
                             w_group_stride=stride)
        m.moe_grouped_linear(h, B * k, None, 1, offsets, E, pool.data_ptr() + 4 * H * I, None, y, B * k, H, I,
                             w_group_stride=stride)
        m.moe_linear(x, dense, None, None, hd, B, I, H, act=m.MOE_ACT_SILU, gated=True)
        m.moe_linear(hd, down, None, None, yd, B, H, I)
        m.moe_combine(y, B * k, pos, w, yd, out, B, k, H)

    x.copy_(normal(g, B, H))
    step()
    torch.cuda.synchronize()
    graph = None
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
    for turn in range(3):
        x.copy_(normal(g, B, H))
        out.fill_(float("nan"))
        if graph:
            graph.replay()
        else:
            step()
        torch.cuda.synchronize()
        want = ref.group(ids.cpu().numpy(), E)
        assert np.array_equal(offsets.cpu().numpy(), want[0])
        assert np.array_equal(order.cpu().numpy(), want[1]) and np.array_equal(pos.cpu().numpy(), want[2])
        rows = torch.from_numpy(want[1] // k).cuda().long()
        hh, hy = ref.product(x, dense, None, "silu", True, chain(H, True))
        ref.check(hd, hh, hy, BF16)
        ref.check(yd, *ref.product(hd, down, None, "none", False, chain(I, True)), BF16)
        total = yd.double()
        size = total.abs()
        for e in range(E):
            lo, hi = want[0][e], want[0][e + 1]
            if lo < hi:
                gu = pool[e, :2 * H * I].view(2 * I, H)
                dn = pool[e, 2 * H * I:blob].view(H, I)
                ref.check(h[lo:hi], *ref.product(x[rows[lo:hi]], gu, None, "silu", True, chain(H, True)), BF16)
                ref.check(y[lo:hi], *ref.product(h[lo:hi], dn, None, "none", False, chain(I, True)), BF16)
        for j in range(k):
            term = y[pos.view(B, k)[:, j].long()].double() * w[:, j:j + 1].double()
            total, size = total + term, size + term.abs()
        assert ((out.double() - total).abs() <= (k + 1) * ref.U * size + 2.0 ** -8 * total.abs() * 1.01 + 1e-30).all()

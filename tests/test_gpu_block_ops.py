"""The operators around the experts on the GPU, against their formulas in 64
bits.  Tolerances are bounds of the fp32 operations (u = 2^-24) and of one
rounding to the output's type; conversions to 4 bits are compared bit for bit."""
import numpy as np
import pytest
import torch

from tests import block_ref as ref

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module")
def m():
    import expert_slot_cache_lru_gb300 as mod
    return mod


def dev(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda()
    return t if dtype is None else t.to(dtype)


def f64(t):
    return t.double().cpu().numpy()


def half_ulp(dtype):
    return 2.0 ** -8 if dtype == torch.bfloat16 else U


def strided(t, stride, offset=0):
    """A copy of the rows of t inside a larger buffer (the rest holds NaN)."""
    big = torch.full((t.shape[0] * stride + offset,), float("nan"), dtype=t.dtype, device="cuda")
    v = big[offset:].view(t.shape[0], stride)[:, :t.shape[1]]
    v.copy_(t)
    return v


# ------------------------------------------------------------------ block norm

def norm_case(m, B, H, res="bf16", post=True, gate="none", alpha=1.0, offset=0.0, pre=True, y=True,
              h_out=True, pad=0, off=0, alias=False, seed=0, spread=3.0):
    r = np.random.default_rng([seed, B, H])
    rt = torch.bfloat16 if res == "bf16" else torch.float32
    bf = torch.bfloat16
    S = H + pad
    mk = lambda t: strided(t, S, off)  # noqa: E731
    h = mk(dev(r.normal(0, spread, (B, H)), rt))
    yt = mk(dev(r.normal(0, 1, (B, H)), bf)) if y else None
    pw = dev(r.normal(1 - offset, 0.2, H), bf) if post and y else None
    qw = dev(r.normal(1 - offset, 0.2, H), bf) if pre else None
    kind, gt, gs = m.MOE_GATE_NONE, None, 0
    if gate != "none":
        rows = gate.endswith("rows")
        kind = m.MOE_GATE_SIGMOID if gate.startswith("sigmoid") else m.MOE_GATE_LINEAR
        gt = mk(dev(r.normal(0, 1, (B, H)), bf)) if rows else dev(r.normal(0, 1, H), bf)
        gs = S if rows else 0
    want_h, want_x, size = ref.block_norm(
        f64(h), f64(yt) if y else None, f64(pw) if pw is not None else None,
        f64(gt) if gt is not None else None, gate.split("_")[0], float(np.float32(alpha)),
        f64(qw) if pre else None, offset, float(np.float32(1e-6)))
    ho = h if alias else mk(torch.zeros(B, H, dtype=rt, device="cuda")) if h_out else None
    xo = (yt if alias and y else mk(torch.zeros(B, H, dtype=bf, device="cuda"))) if pre else None
    m.moe_block_norm(h, yt, pw, gt, qw, ho, xo, B, H,
                     res_dtype=m.MOE_T_BF16 if res == "bf16" else m.MOE_T_F32, gate_kind=kind,
                     alpha=alpha, w_offset=offset, eps=1e-6, h_stride=S, y_stride=S, gate_stride=gs,
                     h_out_stride=S, x_out_stride=S)
    torch.cuda.synchronize()
    # a sum of H squares in at most H/256 + 13 dependent additions, halved by the
    # root, and at most 8 more roundings per term
    c = ((H / 256 + 13) / 2 + 8) * U
    if ho is not None:
        err = np.abs(f64(ho) - want_h)
        assert (err <= half_ulp(rt) * np.abs(want_h) * 1.01 + c * size).all(), err.max()
    if pre:
        inv = np.abs(want_x) / np.maximum(np.abs(want_h), 1e-300)
        err = np.abs(f64(xo) - want_x)
        assert (err <= 2.0 ** -8 * np.abs(want_x) * 1.01 + 2 * c * size * inv + 2.0 ** -133).all(), err.max()


@pytest.mark.parametrize("H", [1, 2, 7, 8, 31, 64, 255, 256, 1000, 2048, 2056, 4095, 4096, 8192, 16384,
                               32761, 32768])
def test_norm_widths(m, H):
    norm_case(m, 3, H)


@pytest.mark.parametrize("res", ["bf16", "f32"])
@pytest.mark.parametrize("gate", ["none", "linear", "sigmoid", "linear_rows", "sigmoid_rows"])
@pytest.mark.parametrize("post,offset", [(True, 0.0), (False, 0.0), (True, 1.0)])
def test_norm_forms(m, res, gate, post, offset):
    norm_case(m, 5, 1032, res=res, gate=gate, post=post, offset=offset, alpha=0.37)


@pytest.mark.parametrize("kw", [
    dict(y=False), dict(pre=False), dict(h_out=False), dict(alias=True), dict(alias=True, res="f32"),
    dict(pad=8), dict(pad=1, gate="linear_rows"), dict(pad=24, off=3, res="f32"),
    dict(pad=16, off=8, gate="sigmoid_rows"), dict(off=1)])
@pytest.mark.parametrize("B,H", [(1, 2048), (600, 512), (37, 777)])
def test_norm_arguments(m, kw, B, H):
    norm_case(m, B, H, **kw)


def test_norm_many_rows(m):
    norm_case(m, 70000, 24, gate="linear_rows", post=True)


@pytest.mark.parametrize("kw", [
    dict(alias=True), dict(alias=True, gate="sigmoid_rows"), dict(gate="sigmoid", offset=1.0, alpha=0.3),
    dict(gate="linear", post=False), dict(y=False), dict(pre=False, gate="linear_rows"),
    dict(h_out=False, pad=8), dict(res="f32", alias=True, gate="linear_rows")])
@pytest.mark.parametrize("B,H", [(1300, 2048), (500, 8192), (5001, 520), (700, 4104), (33, 2047), (19, 8175),
                                 (50, 1002), (9, 13), (17, 8177)])
def test_norm_more_rows_than_fit_at_once(m, kw, B, H):
    norm_case(m, B, H, **kw)


def test_norm_zero_rows_and_extremes(m):
    """A row of zeros stays zero (eps carries the root); a NaN and an infinity
    stay in their own rows."""
    H = 2048
    h = torch.zeros(4, H, device="cuda")
    h[1], h[2, 5], h[3, 7] = 1e-3, float("nan"), float("inf")
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    ho, xo = torch.empty_like(h), torch.empty(4, H, dtype=torch.bfloat16, device="cuda")
    y = torch.zeros(4, H, dtype=torch.bfloat16, device="cuda")
    m.moe_block_norm(h, y, w, None, w, ho, xo, 4, H, res_dtype=m.MOE_T_F32)
    assert not xo[0].any() and not ho[0].any()
    assert abs(xo[1].float().mean().item() - 1e-3 / (1e-6 + 1e-6) ** 0.5) < 0.01
    assert xo[2].isnan().all() and ho[2].isnan().sum() == 1
    assert ho[3, 7] == float("inf") and xo[3, 7].isnan() and not xo[3, :7].any()


def test_norm_offsets_past_32_bits(m):
    """Rows beyond 2^31 elements: the last rows come out as when they are alone."""
    H, B = 8192, 262400
    h = torch.empty(B, H, dtype=torch.bfloat16, device="cuda")
    h.normal_(generator=torch.Generator(device="cuda").manual_seed(1))
    w = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    x = torch.empty_like(h)
    m.moe_block_norm(h, h, w, None, w, None, x, B, H)
    few = torch.empty(3, H, dtype=torch.bfloat16, device="cuda")
    m.moe_block_norm(h[-3:], h[-3:], w, None, w, None, few, 3, H)
    # another kernel sums in another order: a bf16 step at most
    assert ((x[-3:].float() - few.float()).abs() <= 2.0 ** -7 * few.float().abs()).all()


# ------------------------------------------------------------------ router

FORMS = [
    dict(score="softmax"), dict(score="sigmoid"), dict(score="softmax", renorm=False, scale=2.5),
    dict(score="sigmoid", bias=True, scale=2.5), dict(score="softmax", bias=True, renorm=False),
    dict(score="sigmoid", bias=True, groups=4, topk_groups=2, group_top=2),
    dict(score="softmax", groups=4, topk_groups=1, group_top=1, renorm=False),
    dict(score="softmax", groups=2, topk_groups=1, group_top=2),
    dict(score="sigmoid", bias=True, groups=4, topk_groups=3, group_top=1),
]


def check_choice(ids, w, z, k, bias, kw):
    want_ids, want_w, _ = ref.route(z, k, bias=bias, **kw)
    assert np.array_equal(ids, want_ids)
    # exp to 2 ulp, a sum of at most 32 + 5 dependent additions, a division, the
    # sum of k picks and its division, the scale: under 64 roundings
    assert (np.abs(w - want_w) <= 64 * U * np.abs(want_w) + 1e-37).all()


def clear_logits(r, B, E, k, bias, kw):
    """Logits whose different choices differ by more than 1e-6 (equal ones may
    occur), sixteen times fp32's spacing at 1, so that fp32 ranks them alike."""
    z = np.round(r.normal(0, 2, (B, E)) * 64) / 64
    for _ in range(200):
        bad = [b for b in range(B) if ref.route(z[b:b + 1], k, bias=bias, **kw)[2] < 1e-6]
        if not bad:
            return z
        z[bad] = np.round(r.normal(0, 2, (len(bad), E)) * 64) / 64
    raise AssertionError("no clear rows")


def split(kw):
    kw = dict(kw)
    return kw.pop("bias", False), kw


def c_args(m, kw):
    a = {k: v for k, v in kw.items() if k != "score"}
    if "groups" in a:
        a["n_groups"] = a.pop("groups")
    return dict(a, score=m.MOE_SCORE_SOFTMAX if kw["score"] == "softmax" else m.MOE_SCORE_SIGMOID)


@pytest.mark.parametrize("form", range(len(FORMS)))
@pytest.mark.parametrize("E,k", [(8, 1), (16, 4), (60, 6), (64, 8), (128, 8), (160, 6), (256, 8),
                                 (512, 10), (1000, 4), (1024, 32), (1032, 8), (4096, 2)])
def test_route_logits(m, E, k, form):
    has_bias, kw = split(FORMS[form])
    r = np.random.default_rng([E, k, form])
    B = 9
    bias = r.integers(-60, 61, E).astype(np.float32) * np.float32(0.001) if has_bias else None
    z = clear_logits(r, B, E, k, None if bias is None else bias.astype(np.float64), kw)
    for dtype, code in ((torch.float32, m.MOE_T_F32), (torch.bfloat16, m.MOE_T_BF16)):
        zd = strided(dev(z, torch.float32).to(dtype), E + 5)
        if dtype == torch.bfloat16 and ref.route(f64(zd), k, bias=bias, **kw)[2] < 1e-6:
            continue  # rounded to bf16, two choices came closer than fp32 tells apart
        ids = torch.full((B, k), -7, dtype=torch.int32, device="cuda")
        w = torch.full((B, k), -7.0, device="cuda")
        m.moe_route_logits(zd, code, None if bias is None else dev(bias), B, E, k, ids, w,
                           logits_stride=E + 5, **c_args(m, kw))
        check_choice(ids.cpu().numpy(), f64(w), f64(zd),
                     k, None if bias is None else bias.astype(np.float64), kw)


@pytest.mark.parametrize("E", [8, 64, 256, 1024, 1536])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("has_bias", [False, True])
@pytest.mark.parametrize("groups", [1, 4])
def test_route_masks_and_ties(m, E, score, has_bias, groups):
    """Rows masked whole or nearly, ties everywhere, NaN, infinities, signed zeros."""
    inf, nan, k = np.inf, np.nan, 6
    z = np.zeros((10, E))
    z[0] = -inf                      # nothing left
    z[1], z[1, E - 1] = nan, 1.0     # one left
    z[2], z[2, [1, 2]] = -inf, 0.5   # two left, tied
    z[4] = -0.0
    z[4, 3] = 0.0                    # signed zeros tie
    z[5, [E - 1, 0]] = inf           # two infinities share a softmax
    z[6, 1] = nan
    z[6, 2] = -inf
    z[7] = -np.finfo(np.float32).max  # the type's lowest value is a number
    z[7, E // 2] = -3e38
    z[8] = np.arange(E) % 3
    z[9] = -np.arange(E) * 0.5
    bias = np.zeros(E, np.float32) if has_bias else None
    if has_bias:
        bias[E // 4] = -inf          # masks through the bias
        bias[E // 4 + 1] = nan
    kw = dict(score=score, groups=groups, topk_groups=max(1, groups // 2), group_top=1, renorm=True)
    ids = torch.empty(10, k, dtype=torch.int32, device="cuda")
    w = torch.empty(10, k, device="cuda")
    m.moe_route_logits(dev(z, torch.float32), m.MOE_T_F32, None if bias is None else dev(bias), 10, E,
                       k, ids, w, **c_args(m, kw))
    zz = dev(z, torch.float32)
    check_choice(ids.cpu().numpy(), f64(w), f64(zz), k, None if bias is None else bias.astype(np.float64), kw)
    assert (ids[0] == -1).all() and not w[0].any()


ROUTE_SIZES = [(1, 2048, 256, 8), (1, 64, 16, 2), (1, 2047, 60, 4), (3, 4096, 128, 8), (8, 512, 1000, 4),
               (16, 2048, 512, 10), (17, 2048, 256, 8), (33, 1000, 160, 6), (64, 2048, 384, 8),
               (127, 520, 64, 6), (129, 2056, 1024, 2), (600, 2048, 1024, 2), (5, 31, 3, 1),
               (257, 8192, 256, 8), (300, 264, 2048, 8), (1000, 4096, 256, 8)]


@pytest.mark.parametrize("B,H,E,k", ROUTE_SIZES)
@pytest.mark.parametrize("pad", [0, 1, 8])
def test_route(m, B, H, E, k, pad):
    r = np.random.default_rng([B, H, E, k])
    x = strided(dev(r.normal(0, 1, (B, H)), torch.bfloat16), H + pad)
    wr = dev(r.normal(0, H ** -0.5, (E, H)), torch.bfloat16)
    bias = dev((r.integers(-60, 61, E) * 0.001).astype(np.float32))
    z = torch.full((B, E), float("nan"), device="cuda")
    ids = torch.empty(B, k, dtype=torch.int32, device="cuda")
    w = torch.empty(B, k, device="cuda")
    st = torch.zeros(1, dtype=torch.int64, device="cuda")
    m.moe_route(x, wr, bias, B, H, E, k, z, ids, w, score=m.MOE_SCORE_SIGMOID, renorm=True, scale=2.5,
                x_stride=H + pad, d_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    want = x.double() @ wr.double().T
    size = x.double().abs() @ wr.double().abs().T
    # exact products; at most H / 16 + 40 dependent fp32 additions, each of which
    # may truncate (2 u)
    assert ((z.double() - want).abs() <= (H / 16 + 40) * 2 * U * size).all()
    # the choice is exact for the logits that came back
    zz = f64(z)
    kw = dict(score="sigmoid", renorm=True, scale=2.5)
    want_ids, want_w, _ = ref.route(zz, k, bias=f64(bias), **kw)
    got = ids.cpu().numpy()
    _, c = ref.choice(zz, "sigmoid", f64(bias))
    for b in np.nonzero((got != want_ids).any(1))[0]:  # only where fp32 cannot tell two choices apart
        assert np.abs(c[b][got[b]] - c[b][want_ids[b]]).max() < 4 * U, b
    same = (got == want_ids).all(1)
    assert same.mean() > 0.99 or B < 100
    assert (np.abs(f64(w) - want_w)[same] <= 64 * U * np.abs(want_w)[same] + 1e-37).all()


@pytest.mark.parametrize("B,H,E", [(20500, 256, 256), (40000, 128, 100), (30001, 72, 64), (20000, 512, 700)])
def test_route_more_tiles_than_sms(m, B, H, E):
    """Every logit of products whose CTAs take several tiles each, and each row's best expert."""
    r = np.random.default_rng([B, H, E])
    x = dev(r.normal(0, 1, (B, H)), torch.bfloat16)
    wr = dev(r.normal(0, H ** -0.5, (E, H)), torch.bfloat16)
    z = torch.full((B, E), float("nan"), device="cuda")
    ids = torch.empty(B, 1, dtype=torch.int32, device="cuda")
    w = torch.empty(B, 1, device="cuda")
    m.moe_route(x, wr, None, B, H, E, 1, z, ids, w, renorm=False)
    want = x.double() @ wr.double().T
    assert ((z.double() - want).abs() <= (H / 16 + 40) * 2 * U * (x.double().abs() @ wr.double().abs().T)).all()
    assert torch.equal(z.gather(1, ids.long()), z.max(1, keepdim=True).values)
    p = torch.softmax(z.double(), 1).gather(1, ids.long())
    assert ((w.double() - p).abs() <= 64 * U * p).all()


def test_route_twice_the_same_and_in_a_graph(m):
    r = np.random.default_rng(5)
    for B, H, E, k in [(1, 2048, 256, 8), (40, 2048, 256, 8), (600, 2048, 1024, 2)]:
        x = dev(r.normal(0, 1, (B, H)), torch.bfloat16)
        wr = dev(r.normal(0, H ** -0.5, (E, H)), torch.bfloat16)
        outs = [(torch.empty(B, E, device="cuda"), torch.empty(B, k, dtype=torch.int32, device="cuda"),
                 torch.empty(B, k, device="cuda")) for _ in range(2)]
        m.moe_route(x, wr, None, B, H, E, k, *outs[0])
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            m.moe_route(x, wr, None, B, H, E, k, *outs[1])
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(*outs):
            assert torch.equal(a, b)


# ------------------------------------------------------------------ 4-bit conversions

def fmt_of(m, nv):
    return m.MOE_W_NVFP4 if nv else m.MOE_W_MXFP4


def quantize(m, x, nv, g, stride=0):
    B, K = x.shape
    codes = torch.full((B, K // 2), 0xEE, dtype=torch.uint8, device="cuda")
    scales = torch.full((B, K // (16 if nv else 32)), 0xEE, dtype=torch.uint8, device="cuda")
    gd = None if g is None else torch.tensor([g], dtype=torch.float32, device="cuda")
    m.moe_fp4_quantize(fmt_of(m, nv), x, m.MOE_T_BF16 if x.dtype == torch.bfloat16 else m.MOE_T_F32, B, K,
                       gd, codes, scales, src_stride=stride)
    return codes, scales, gd


@pytest.mark.parametrize("nv,g", [(True, None), (True, 1.0), (True, 0.0421 / 2688), (True, 0.25),
                                  (False, None)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,K,pad", [(1, 32, 0), (1, 2048, 0), (3, 96, 1), (7, 160, 4), (33, 512, 8),
                                     (1000, 64, 0), (129, 2080, 16), (64, 8192, 0)])
def test_quantize_bits(m, nv, dtype, B, K, pad, g):
    r = np.random.default_rng([B, K, pad])
    std = np.exp(r.uniform(-3, 3, (B, 1))) * (1.0 if g is None else g * 300)
    x = strided(dev(r.normal(0, 1, (B, K)) * std, torch.float32).to(dtype), K + pad)
    codes, scales, gd = quantize(m, x, nv, g, K + pad)
    want_c, want_s = ref.quantize(x.float().cpu().numpy(), nv, g)
    assert np.array_equal(scales.cpu().numpy(), want_s)
    assert np.array_equal(codes.cpu().numpy(), want_c)
    # and back: (code * s) * g, one rounding each
    for dt, code in ((torch.float32, m.MOE_T_F32), (torch.bfloat16, m.MOE_T_BF16)):
        v = strided(torch.zeros(B, K, dtype=dt, device="cuda"), K + pad)
        m.moe_fp4_dequantize(fmt_of(m, nv), codes, scales, gd, B, K, v, code, dst_stride=K + pad)
        base = ref.decode(want_c, want_s, nv).astype(np.float32) * np.float32(1.0 if g is None else g)
        assert torch.equal(v, dev(base).to(dt))


@pytest.mark.parametrize("nv", [True, False])
def test_quantize_special_blocks(m, nv):
    blk = 16 if nv else 32
    x = np.zeros((1, 12 * blk), np.float32)
    b = x.reshape(12, blk)
    b[11, 3] = -0.0
    b[2] = 1e-30                     # the scale rounds to zero (NVFP4)
    b[3, 0], b[3, 1] = np.nan, 1.0
    b[4, 0], b[4, 1], b[4, 2] = np.inf, 3.0, -np.inf
    b[5, :8] = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5]   # exact ties
    b[6, :8] = [-6, -0.25, -0.75, -1.25, -1.75, -2.5, -3.5, -5]
    b[7] = 3e38
    b[8] = 1e-45                     # the smallest denormal
    b[9, 0] = 2688.0
    b[10, 0], b[10, 1] = 7.999, 0.5   # beyond 6 * 2^0 for MXFP4: saturates
    b[11, 0], b[11, 1] = 2.0, 1.9375  # and a negative zero
    t = dev(x)
    codes, scales, gd = quantize(m, t, nv, None)
    want_c, want_s = ref.quantize(x, nv)
    assert np.array_equal(scales.cpu().numpy(), want_s)
    assert np.array_equal(codes.cpu().numpy(), want_c)
    v = torch.empty(1, 12 * blk, device="cuda")
    m.moe_fp4_dequantize(fmt_of(m, nv), codes, scales, None, 1, 12 * blk, v, m.MOE_T_F32)
    v = v.view(12, blk).cpu().numpy()
    assert np.isnan(v[3]).all() and not np.isnan(np.delete(v, 3, 0)).any()
    assert np.signbit(v[11, 3]) and not np.signbit(v[11, 4])
    assert v[5, :8].tolist() == [6, 0, 1, 1, 2, 2, 4, 4]
    # an infinity takes code 6 under the largest scale: 2688, or 6 * 2^126, which fp32 does not hold
    assert v[4, 0] == -v[4, 2] == (2688 if nv else np.inf)


@pytest.mark.parametrize("nv", [True, False])
def test_every_code_and_scale_reads_back(m, nv):
    blk = 16 if nv else 32
    scales = torch.arange(256, dtype=torch.uint8, device="cuda").repeat_interleave(2).view(1, -1)
    n = scales.shape[1] * blk
    codes = torch.arange(n // 2, device="cuda").to(torch.uint8).view(1, -1)
    v = torch.empty(1, n, device="cuda")
    m.moe_fp4_dequantize(fmt_of(m, nv), codes, scales, None, 1, n, v, m.MOE_T_F32)
    want = ref.decode(codes.cpu().numpy(), scales.cpu().numpy(), nv)
    assert np.array_equal(f64(v), want.astype(np.float32).astype(np.float64), equal_nan=True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B,K,pad", [(1, 1, 0), (3, 77, 2), (600, 2048, 0)])
def test_global_scale(m, dtype, B, K, pad):
    r = np.random.default_rng([B, K])
    x = strided(dev(r.normal(0, 1, (B, K)), dtype), K + pad)
    code = m.MOE_T_BF16 if dtype == torch.bfloat16 else m.MOE_T_F32
    g = torch.full((1,), 7.0, device="cuda")
    m.moe_fp4_global_scale(x, code, B, K, g, src_stride=K + pad)
    assert g.item() == np.float32(x.float().abs().max().item()) / np.float32(2688)
    x[0, 0] = float("inf")
    if K > 1:
        x[0, 1] = float("nan")
        m.moe_fp4_global_scale(x, code, B, K, g, src_stride=K + pad)
        assert g.item() == np.float32(f64(x)[np.isfinite(f64(x))].__abs__().max()) / np.float32(2688)
    x.zero_()
    m.moe_fp4_global_scale(x, code, B, K, g, src_stride=K + pad)
    assert g.item() == 1.0


def test_quantize_offsets_past_32_bits(m):
    B, K = 70000, 32768
    x = torch.empty(B, K, dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=torch.Generator(device="cuda").manual_seed(2))
    codes, scales, g = quantize(m, x, True, 0.01)
    c, s, _ = quantize(m, x[-2:].contiguous(), True, 0.01)
    assert torch.equal(codes[-2:], c) and torch.equal(scales[-2:], s)
    m.moe_fp4_dequantize(m.MOE_W_NVFP4, codes, scales, g, B, K, x, m.MOE_T_BF16)
    v = torch.empty(2, K, dtype=torch.bfloat16, device="cuda")
    m.moe_fp4_dequantize(m.MOE_W_NVFP4, c, s, g, 2, K, v, m.MOE_T_BF16)
    assert torch.equal(x[-2:], v)


# ------------------------------------------------------------------ 4-bit product

LINEAR = [(1, 16, 32), (1, 130, 64), (1, 4096, 2048), (2, 1000, 512), (5, 257, 2080), (8, 512, 4096),
          (16, 2048, 96), (17, 384, 1024), (33, 4097, 256), (64, 1536, 2048), (100, 640, 288),
          (128, 128, 256), (129, 255, 2080), (200, 2048, 512), (255, 300, 320), (256, 256, 4096),
          (600, 1536, 2048), (513, 1030, 544), (1000, 8, 64), (2048, 2048, 2048), (1930, 2000, 544),
          (700, 7001, 96), (5000, 5000, 160), (20, 70000, 64), (3000, 2500, 64),
          (40, 20000, 320), (64, 19500, 512)]


def linear_case(m, nv, B, N, K, dtype, pad=0, seed=0, g=True):
    r = np.random.default_rng([seed, B, N, K])
    blk = 16 if nv else 32
    lo, hi = (0x20, 0x40) if nv else (118, 130)
    xc, wc = (r.integers(0, 256, (n, K // 2)).astype(np.uint8) for n in (B, N))
    xs, ws = (r.integers(lo, hi, (n, K // blk)).astype(np.uint8) for n in (B, N))
    xg, wg = (0.75, 0.011) if nv and g else (None, None)
    out = strided(torch.zeros(B, N, dtype=dtype, device="cuda"), N + pad)
    gd = [None if v is None else torch.tensor([v], device="cuda") for v in (xg, wg)]
    st = torch.zeros(1, dtype=torch.int64, device="cuda")
    m.moe_fp4_linear(fmt_of(m, nv), dev(xc), dev(xs), gd[0], dev(wc), dev(ws), gd[1], B, N, K, out,
                     m.MOE_T_BF16 if dtype == torch.bfloat16 else m.MOE_T_F32, out_stride=N + pad,
                     d_status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    x, w = dev(ref.decode(xc, xs, nv, xg)), dev(ref.decode(wc, ws, nv, wg))
    want, size = x @ w.T, x.abs() @ w.abs().T
    # exact products; at most K / 32 + 40 dependent fp32 additions, each of which
    # may truncate (2 u); the product of the global scales and its product: 2 u
    tol = ((K / 32 + 40) * 2 * U) * size + 1.01 * half_ulp(dtype) * want.abs()
    err = (out.double() - want).abs()
    assert (err <= tol).all(), ((err / tol).max().item(), err.max().item())
    if pad:
        whole = out.as_strided((B, N + pad), (N + pad, 1))
        assert whole[:, N:].isnan().all()  # nothing written between the rows


@pytest.mark.parametrize("nv", [True, False])
@pytest.mark.parametrize("B,N,K", LINEAR)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_linear(m, nv, B, N, K, dtype):
    linear_case(m, nv, B, N, K, dtype)


@pytest.mark.parametrize("B,N,K", [(1, 300, 128), (40, 300, 512), (300, 300, 512)])
@pytest.mark.parametrize("pad", [1, 4, 8])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_linear_strided_output(m, B, N, K, pad, dtype):
    linear_case(m, True, B, N, K, dtype, pad=pad, g=False)


def test_linear_offsets_past_32_bits(m):
    """An output beyond 2^31 elements: its last rows as when they are alone."""
    B, N, K = 36000, 60000, 64
    r = np.random.default_rng(9)
    xc, wc = (dev(r.integers(0, 256, (n, K // 2)).astype(np.uint8)) for n in (B, N))
    xs, ws = (dev(r.integers(0x28, 0x38, (n, K // 16)).astype(np.uint8)) for n in (B, N))
    out = torch.empty(B, N, dtype=torch.bfloat16, device="cuda")
    m.moe_fp4_linear(m.MOE_W_NVFP4, xc, xs, None, wc, ws, None, B, N, K, out, m.MOE_T_BF16)
    x = dev(ref.decode(xc[-2:].cpu().numpy(), xs[-2:].cpu().numpy(), True))
    w = dev(ref.decode(wc.cpu().numpy(), ws.cpu().numpy(), True))
    want = x @ w.T
    assert ((out[-2:].double() - want).abs() <= 1.01 * 2.0 ** -8 * want.abs() + 84 * U * (x.abs() @ w.abs().T)).all()


@pytest.mark.parametrize("nv", [True, False])
@pytest.mark.parametrize("B", [3, 300])
def test_linear_nan_scale_stays_in_its_row(m, nv, B):
    """A NaN block scale of x spoils that row of the output and no other; NaN
    scales after the last row or block of a bank are never read."""
    K, N, blk = 544, 200, 16 if nv else 32
    one = 0x38 if nv else 127
    xs = torch.full((B + 1, K // blk), one, dtype=torch.uint8, device="cuda")
    ws = torch.full((N + 1, K // blk), one, dtype=torch.uint8, device="cuda")
    xs[B], ws[N] = 0x7F if nv else 0xFF, 0x7F if nv else 0xFF
    xs[1, K // blk - 1] = 0x7F if nv else 0xFF
    xc = torch.full((B, K // 2), 0x22, dtype=torch.uint8, device="cuda")  # all ones
    wc = torch.full((N, K // 2), 0x22, dtype=torch.uint8, device="cuda")
    out = torch.empty(B, N, device="cuda")
    m.moe_fp4_linear(fmt_of(m, nv), xc, xs, None, wc, ws, None, B, N, K, out, m.MOE_T_F32)
    assert out[1].isnan().all()
    assert (out[torch.arange(B) != 1] == K).all()


def test_linear_of_quantized_data(m):
    """bf16 x and w through the converter and the product: the error is that of
    4 bits (half a step of at most a third of a block's maximum, averaged)."""
    r = np.random.default_rng(3)
    for nv in (True, False):
        x = dev(r.normal(0, 1, (50, 2048)), torch.bfloat16)
        w = dev(r.normal(0, 0.02, (300, 2048)), torch.bfloat16)
        g = [None, None]
        if nv:
            g = [torch.empty(1, device="cuda") for _ in range(2)]
            m.moe_fp4_global_scale(x, m.MOE_T_BF16, 50, 2048, g[0])
            m.moe_fp4_global_scale(w, m.MOE_T_BF16, 300, 2048, g[1])
        bank = []
        for t, gt in ((x, g[0]), (w, g[1])):
            c, s, _ = quantize(m, t, nv, None if gt is None else gt.item())
            bank += [c, s, gt]
        out = torch.empty(50, 300, device="cuda")
        m.moe_fp4_linear(fmt_of(m, nv), *bank, 50, 300, 2048, out, m.MOE_T_F32)
        want = x.double() @ w.double().T
        assert ((out.double() - want).norm() / want.norm()).item() < 0.25


def test_linear_on_a_side_stream_and_in_a_graph(m):
    r = np.random.default_rng(4)
    for B, N, K in [(1, 4096, 2048), (300, 512, 1024)]:
        a = [dev(r.integers(0, 256, (n, K // 2)).astype(np.uint8)) for n in (B, N)]
        sc = [dev(r.integers(0x28, 0x38, (n, K // 16)).astype(np.uint8)) for n in (B, N)]
        outs = [torch.zeros(B, N, device="cuda") for _ in range(3)]
        call = lambda o, st: m.moe_fp4_linear(m.MOE_W_NVFP4, a[0], sc[0], None, a[1], sc[1], None, B, N,  # noqa: E731
                                              K, o, m.MOE_T_F32, stream=st)
        call(outs[0], None)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        call(outs[1], s)
        g = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(g, stream=s):
            call(outs[2], s)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])

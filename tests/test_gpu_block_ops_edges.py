"""The operators around the experts where buffers are used again, calls follow each
other without a stop, and values or sizes are extreme.  Tolerances as in
test_gpu_block_ops.py."""
import numpy as np
import pytest
import torch

from tests import block_ref as ref
from tests.test_gpu_block_ops import U, c_args, check_choice, dev, fmt_of, half_ulp, m  # noqa: F401  (m: the library)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ 4-bit product

def banks(r, nv, rows, K):
    lo, hi = (0x20, 0x40) if nv else (118, 130)
    return (dev(r.integers(0, 256, (rows, K // 2)).astype(np.uint8)),
            dev(r.integers(lo, hi, (rows, K // (16 if nv else 32))).astype(np.uint8)))


@pytest.mark.parametrize("nv", [True, False])
@pytest.mark.parametrize("B,N,K", [(129, 40000, 256), (257, 40000, 512), (300, 40000, 64), (1025, 16000, 256),
                                   (8193, 2048, 256), (8225, 2048, 512), (4129, 8200, 128), (5000, 5000, 160)])
def test_linear_bf16_tiles_with_warps_past_the_last_row(m, nv, B, N, K):  # noqa: F811
    """CTAs that go from whole tiles to tiles some of whose warps have no rows: bf16
    results, which leave through two buffers in turn, are the fp32 results (which wait
    for each copy) rounded, everywhere and every time."""
    r = np.random.default_rng([B, N, K])
    xc, xs = banks(r, nv, B, K)
    wc, ws = banks(r, nv, N, K)
    f32 = torch.empty(B, N, device="cuda")
    m.moe_fp4_linear(fmt_of(m, nv), xc, xs, None, wc, ws, None, B, N, K, f32, m.MOE_T_F32)
    x = dev(ref.decode(xc[-2:].cpu().numpy(), xs[-2:].cpu().numpy(), nv))
    w = dev(ref.decode(wc.cpu().numpy(), ws.cpu().numpy(), nv))
    assert ((f32[-2:].double() - x @ w.T).abs() <= (K / 32 + 40) * 2 * U * (x.abs() @ w.abs().T)).all()
    for _ in range(5):
        out = torch.full((B, N), float("nan"), dtype=torch.bfloat16, device="cuda")
        m.moe_fp4_linear(fmt_of(m, nv), xc, xs, None, wc, ws, None, B, N, K, out, m.MOE_T_BF16)
        assert torch.equal(out, f32.bfloat16())


# ------------------------------------------------------------------ chains without a stop

def chain(step, n, sources):
    """step(source) runs calls that go through one set of buffers and returns fresh
    outputs; n rounds over the sources in turn, enqueued without a stop, give what each
    source gives alone."""
    want = []
    for s in sources:
        torch.cuda.synchronize()
        want.append(step(s))
        torch.cuda.synchronize()
    got = [step(sources[i % len(sources)]) for i in range(n)]
    torch.cuda.synchronize()
    for i, outs in enumerate(got):
        for a, b in zip(outs, want[i % len(sources)]):
            assert torch.equal(a, b), i


@pytest.mark.parametrize("nv", [True, False])
@pytest.mark.parametrize("B,K,pad", [(1, 512, 0), (64, 2048, 0), (64, 2048, 1), (600, 2080, 0), (4096, 1024, 0)])
def test_banks_rewritten_between_calls(m, nv, B, K, pad):  # noqa: F811
    """Two sources in turn through one code bank: bf16 to fp32 and back."""
    r = np.random.default_rng([B, K])
    src = [dev(r.normal(0, s, (B, K + pad)), torch.bfloat16) for s in (1.0, 3.0)]
    codes = torch.empty(B, K // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(B, K // (16 if nv else 32), dtype=torch.uint8, device="cuda")
    f = fmt_of(m, nv)

    def step(x):
        v, back = torch.empty(B, K, device="cuda"), torch.empty(B, K, dtype=torch.bfloat16, device="cuda")
        m.moe_fp4_quantize(f, x, m.MOE_T_BF16, B, K, None, codes, scales, src_stride=K + pad)
        m.moe_fp4_dequantize(f, codes, scales, None, B, K, v, m.MOE_T_F32)
        m.moe_fp4_quantize(f, v, m.MOE_T_F32, B, K, None, codes, scales)
        m.moe_fp4_dequantize(f, codes, scales, None, B, K, back, m.MOE_T_BF16)
        return v, back

    chain(step, 40, src)


@pytest.mark.parametrize("B,H,E", [(1, 2048, 256), (3, 520, 60), (8, 4096, 64), (40, 2048, 256), (600, 1000, 128),
                                   (5, 2047, 30)])
def test_activations_rewritten_between_calls(m, B, H, E):  # noqa: F811
    """Norm, router, quantise and the 4-bit product through one x and one pair of banks."""
    r = np.random.default_rng([B, H, E])
    bf = torch.bfloat16
    src = [(dev(r.normal(0, 2, (B, H)), bf), dev(r.normal(0, 1, (B, H)), bf)) for _ in range(2)]
    w, router = dev(r.normal(1, 0.1, H), bf), dev(r.normal(0, H ** -0.5, (E, H)), bf)
    bias = dev((r.integers(-60, 61, E) * 0.001).astype(np.float32))
    K = H // 32 * 32
    wc, ws = banks(r, True, 96, K)
    x = torch.empty(B, H, dtype=bf, device="cuda")
    xc = torch.empty(B, K // 2, dtype=torch.uint8, device="cuda")
    xs = torch.empty(B, K // 16, dtype=torch.uint8, device="cuda")

    def step(s):
        z, wt, out = (torch.empty(B, n, device="cuda") for n in (E, 4, 96))
        ids = torch.empty(B, 4, dtype=torch.int32, device="cuda")
        m.moe_block_norm(s[0], s[1], w, None, w, None, x, B, H)
        m.moe_route(x, router, bias, B, H, E, 4, z, ids, wt, score=m.MOE_SCORE_SIGMOID)
        m.moe_fp4_quantize(m.MOE_W_NVFP4, x, m.MOE_T_BF16, B, K, None, xc, xs, src_stride=H)
        m.moe_fp4_linear(m.MOE_W_NVFP4, xc, xs, None, wc, ws, None, B, 96, K, out, m.MOE_T_F32)
        return z, ids, wt, out

    chain(step, 40, src)


def test_router_made_by_the_call_before(m):  # noqa: F811
    """Weights that another call has just written: two routers from 4 bits, in turn."""
    r = np.random.default_rng(11)
    H, E = 512, 64
    src = [banks(r, True, E, H) for _ in range(2)]
    router = torch.empty(E, H, dtype=torch.bfloat16, device="cuda")
    norm_w = router.view(-1)[:H]
    x = {B: dev(r.normal(0, 1, (B, H)), torch.bfloat16) for B in (2, 700)}

    def step(s):
        outs = []
        for B in (2, 700):
            z, w = torch.empty(B, E, device="cuda"), torch.empty(B, 2, device="cuda")
            ids, n = torch.empty(B, 2, dtype=torch.int32, device="cuda"), torch.empty_like(x[B])
            m.moe_fp4_dequantize(m.MOE_W_NVFP4, *s, None, E, H, router, m.MOE_T_BF16)
            m.moe_route(x[B], router, None, B, H, E, 2, z, ids, w)
            m.moe_fp4_dequantize(m.MOE_W_NVFP4, *s, None, E, H, router, m.MOE_T_BF16)
            m.moe_block_norm(x[B], None, None, None, norm_w, None, n, B, H)
            outs += [z, ids, w, n]
        return outs

    chain(step, 40, src)


# ------------------------------------------------------------------ rows near 2^31

MOST = 2 ** 31 - 1


def test_global_scale_of_the_most_rows(m):  # noqa: F811
    x = torch.ones(MOST, 2, dtype=torch.bfloat16, device="cuda")
    g = torch.empty(1, device="cuda")
    for at in (MOST - 1, MOST - 1025, 5):
        x[at, 0], x[at, 1] = 24.0, 99.0  # 99: between the rows
        m.moe_fp4_global_scale(x, m.MOE_T_BF16, MOST, 1, g, src_stride=2)
        assert g.item() == np.float32(24) / np.float32(2688)
        x[at] = 1.0


def test_conversions_of_the_most_rows(m):  # noqa: F811
    """Strided rows of one block each, of which the last and some others are looked at."""
    x = torch.empty(MOST * 17, dtype=torch.bfloat16, device="cuda").view(MOST, 17)
    x.zero_()
    codes = torch.empty(MOST, 8, dtype=torch.uint8, device="cuda")
    scales = torch.empty(MOST, 1, dtype=torch.uint8, device="cuda")
    some = torch.tensor([0, 65534, 65535, 2 ** 30, MOST - 65536, MOST - 65535, MOST - 2, MOST - 1], device="cuda")
    r = np.random.default_rng(1)
    v = dev(r.normal(0, 1, (8, 16)).astype(np.float32)).bfloat16()
    x[some, :16] = v
    m.moe_fp4_quantize(m.MOE_W_NVFP4, x, m.MOE_T_BF16, MOST, 16, None, codes, scales, src_stride=17)
    want_c, want_s = ref.quantize(v.float().cpu().numpy(), True)
    assert np.array_equal(codes[some].cpu().numpy(), want_c) and np.array_equal(scales[some].cpu().numpy(), want_s)
    x[some] = 7.0
    m.moe_fp4_dequantize(m.MOE_W_NVFP4, codes, scales, None, MOST, 16, x, m.MOE_T_BF16, dst_stride=17)
    back = x[some].double().cpu().numpy()
    assert np.array_equal(back[:, :16], ref.decode(want_c, want_s, True).astype(np.float32)) and (back[:, 16] == 7).all()


@pytest.mark.parametrize("nv", [True, False])
def test_linear_of_the_most_weights(m, nv):  # noqa: F811
    one, blk = (0x38, 16) if nv else (127, 32)
    xc = torch.full((1, 16), 0x22, dtype=torch.uint8, device="cuda")  # all ones
    xs = torch.full((1, 32 // blk), one, dtype=torch.uint8, device="cuda")
    wc = torch.zeros(MOST, 16, dtype=torch.uint8, device="cuda")
    ws = torch.full((MOST, 32 // blk), one, dtype=torch.uint8, device="cuda")
    some = torch.tensor([0, 127, 2 ** 30, MOST - 129, MOST - 128, MOST - 1], device="cuda")
    v = np.random.default_rng(2).integers(0, 256, (6, 16)).astype(np.uint8)
    wc[some] = dev(v)
    out = torch.full((1, MOST), float("nan"), dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int64, device="cuda")
    m.moe_fp4_linear(fmt_of(m, nv), xc, xs, None, wc, ws, None, 1, MOST, 32, out, m.MOE_T_BF16, d_status=st)
    assert st.item() == 0
    want = ref.decode(v, np.full((6, 32 // blk), one, np.uint8), nv).sum(1)  # multiples of a half below 192
    assert np.array_equal(out[0, some].double().cpu().numpy(), dev(want).bfloat16().double().cpu().numpy())
    out[0, some] = 0.0
    assert not out.any()


def test_route_of_the_most_rows(m):  # noqa: F811
    x = torch.zeros(MOST, 8, dtype=torch.bfloat16, device="cuda")
    router = torch.ones(1, 8, dtype=torch.bfloat16, device="cuda")
    some = torch.tensor([0, 2 ** 30, MOST - 130, MOST - 1], device="cuda")
    v = dev(np.random.default_rng(3).normal(0, 1, (4, 8)).astype(np.float32)).bfloat16()
    x[some] = v
    z, w = (torch.full((MOST, 1), float("nan"), device="cuda") for _ in range(2))
    ids = torch.full((MOST, 1), -7, dtype=torch.int32, device="cuda")
    m.moe_route(x, router, None, MOST, 8, 1, 1, z, ids, w)
    assert ((z[some].double() - v.double().sum(1, keepdim=True)).abs() <= 41 * 2 * U * v.double().abs().sum(1, keepdim=True)).all()
    z[some] = 0.0
    assert not z.any() and not ids.any() and bool((w == 1).all())


# ------------------------------------------------------------------ router: extreme choices

@pytest.mark.parametrize("E", [8, 64, 256, 1024, 1536])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_groups_whose_sum_passes_fp32(m, E, score):  # noqa: F811
    """group_top 2 with biases of the type's lowest value, a common finite mask: two of
    them add up to less than fp32 holds, and the group still has unmasked experts."""
    low, G, k = -np.finfo(np.float32).max, 4, 6
    gs = E // G
    kw = dict(score=score, groups=G, topk_groups=3, group_top=2, renorm=True)
    r = np.random.default_rng(E)
    z = np.round(r.normal(0, 2, (5, E)) * 64) / 64
    for case in range(4):
        bias = np.zeros(E, np.float32)
        if case == 0:
            bias[:] = low                    # every group
        elif case == 1:
            bias[gs:] = low                  # all but the first
        elif case == 2:
            bias[:gs] = low
            bias[gs:2 * gs] = -np.inf        # truly masked: behind the lowest ones
            bias[2 * gs:3 * gs] = low
        else:
            bias[:] = low
            bias[gs:gs + 2] = -low           # sums beyond the other end
            bias[3 * gs:] = np.nan
        ids = torch.full((5, k), -7, dtype=torch.int32, device="cuda")
        w = torch.full((5, k), -7.0, device="cuda")
        m.moe_route_logits(dev(z, torch.float32), m.MOE_T_F32, dev(bias), 5, E, k, ids, w, **c_args(m, kw))
        # in fp32 the choices under the lowest value are equal: s + low = low
        want = np.full((5, k), -1)
        alive = [g for g in range(G) if not (np.isnan(bias[g * gs]) or bias[g * gs] == -np.inf)]
        best = {g: np.clip(2.0 * np.float64(bias[g * gs]), low, -low) for g in alive}
        kept = sorted(sorted(alive, key=lambda g: (-best[g], g))[:3])
        for b in range(5):
            s, c = ref.choice(z[b:b + 1], score, np.zeros(E))
            choice = np.where(bias == low, low, np.where(bias == -low, -low, c[0] + bias))
            cand = [e for g in kept for e in range(g * gs, (g + 1) * gs)]
            pick = sorted(cand, key=lambda e: (-choice[e], e))[:k]
            want[b, :len(pick)] = pick
            assert ids[b].tolist() == want[b].tolist(), (case, b)
            p = s[0][pick] / s[0][pick].sum()
            assert (np.abs(w[b].double().cpu().numpy()[:len(pick)] - p) <= 64 * U * p + 1e-37).all()


def far_apart(E, lo, hi):
    """Logits of a row from lo to hi, different ones, in multiples of 1/64 (differences are exact in fp32)."""
    return np.round(np.linspace(hi, lo, E) * 64) / 64


@pytest.mark.parametrize("E", [60, 64, 256, 1024, 1536])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("form", ["plain", "bias", "groups"])
def test_route_weights_of_logits_far_apart(m, E, score, renorm, form):  # noqa: F811
    """Scores many powers of ten below the largest are as exact as the largest: the picks' weights
    against the formula, each within a few fp32 roundings of itself."""
    k, r = 16, np.random.default_rng(E)
    z = np.stack([far_apart(E, -80, 0), far_apart(E, -85, 20), r.permutation(far_apart(E, -60, 3)),
                  far_apart(E, -86, -50)])
    kw = dict(score=score, renorm=renorm, scale=1.0)
    bias = None
    if form == "bias":  # 2 more for the experts of smallest score, in different steps
        bias = np.zeros(E, np.float32)
        bias[-20:] = 2 + np.arange(20) * np.float32(0.25)
    if form == "groups":
        kw.update(groups=2, topk_groups=1, group_top=2)
    ids = torch.empty(4, k, dtype=torch.int32, device="cuda")
    w = torch.empty(4, k, device="cuda")
    m.moe_route_logits(dev(z, torch.float32), m.MOE_T_F32, None if bias is None else dev(bias), 4, E, k, ids, w,
                       **c_args(m, kw))
    check_choice(ids.cpu().numpy(), w.double().cpu().numpy(), z, k,
                 None if bias is None else bias.astype(np.float64), kw)


@pytest.mark.parametrize("E", [16, 256, 1536])
@pytest.mark.parametrize("has_bias", [False, True])
def test_route_sigmoids_near_the_smallest_normal_number(m, E, has_bias):  # noqa: F811
    """All logits at -85 to -88.5: scores down to 4e-39, whose shares are still plain numbers."""
    k, z = 4, far_apart(E, -88.5, -85)[None]
    kw = dict(score="sigmoid", renorm=True, scale=2.5)
    bias = np.zeros(E, np.float32) if has_bias else None
    if has_bias:
        bias[-4:] = [4, 3, 2, 1]  # the smallest scores
    ids = torch.empty(1, k, dtype=torch.int32, device="cuda")
    w = torch.empty(1, k, device="cuda")
    m.moe_route_logits(dev(z, torch.float32), m.MOE_T_F32, None if bias is None else dev(bias), 1, E, k, ids, w,
                       **c_args(m, kw))
    check_choice(ids.cpu().numpy(), w.double().cpu().numpy(), z, k,
                 None if bias is None else bias.astype(np.float64), kw)


# ------------------------------------------------------------------ block norm: extreme gates

@pytest.mark.parametrize("res", ["bf16", "f32"])
@pytest.mark.parametrize("rows_gate", [False, True])
@pytest.mark.parametrize("B,H", [(2, 64), (700, 2048), (5, 1002), (3, 8200), (400, 4104)])
def test_norm_sigmoid_gates_far_from_zero(m, res, rows_gate, B, H):  # noqa: F811
    """Gates from -88.5 to 40 on a block output of up to 2e38: terms that count come out as
    exact as the others, down to sigmoids of 4e-39."""
    r = np.random.default_rng([B, H])
    rt = torch.bfloat16 if res == "bf16" else torch.float32
    g = dev(r.uniform(-88.5, 40, (B, H) if rows_gate else (1, H)).astype(np.float32)).bfloat16()
    g[:, 0], g[:, 1] = -88.0, 0.0
    # a term of size 1 or so: 1 / sigmoid(gate) times a normal number
    y = (torch.exp(-g.double()).add(1).expand(B, H) * dev(r.normal(0, 0.5, (B, H)))).clamp(-2e38, 2e38).bfloat16()
    h = dev(r.normal(0, 0.01, (B, H)).astype(np.float32)).to(rt)
    ho, qw = torch.empty_like(h), torch.ones(H, dtype=torch.bfloat16, device="cuda")
    xo = torch.empty(B, H, dtype=torch.bfloat16, device="cuda")
    m.moe_block_norm(h, y, None, g, qw, ho, xo, B, H, res_dtype=m.MOE_T_BF16 if res == "bf16" else m.MOE_T_F32,
                     gate_kind=m.MOE_GATE_SIGMOID, gate_stride=H if rows_gate else 0)
    f64 = lambda t: t.double().cpu().numpy()  # noqa: E731
    want, x, size = ref.block_norm(f64(h), f64(y), None, f64(g), "sigmoid", 1.0, f64(qw), eps=float(np.float32(1e-6)))
    c = ((H / 256 + 13) / 2 + 8) * U  # as test_gpu_block_ops.norm_case
    assert (np.abs(f64(ho) - want) <= half_ulp(rt) * np.abs(want) * 1.01 + c * size).all()
    inv = np.abs(x) / np.maximum(np.abs(want), 1e-300)
    assert (np.abs(f64(xo) - x) <= 2.0 ** -8 * np.abs(x) * 1.01 + 2 * c * size * inv + 2.0 ** -133).all()


@pytest.mark.parametrize("res", ["bf16", "f32"])
@pytest.mark.parametrize("B,H", [(2, 64), (700, 2048), (5, 1002)])
def test_norm_infinite_output_under_a_gate(m, res, B, H):  # noqa: F811
    """An infinity times a sigmoid that is a number stays an infinity."""
    rt = torch.bfloat16 if res == "bf16" else torch.float32
    h = torch.zeros(B, H, dtype=rt, device="cuda")
    y = torch.full((B, H), float("inf"), dtype=torch.bfloat16, device="cuda")
    g = torch.full((B, H), -88.0, dtype=torch.bfloat16, device="cuda")
    m.moe_block_norm(h, y, None, g, None, h, None, B, H, res_dtype=m.MOE_T_BF16 if res == "bf16" else m.MOE_T_F32,
                     gate_kind=m.MOE_GATE_SIGMOID, gate_stride=H)
    assert bool((h == float("inf")).all())


@pytest.mark.parametrize("res", ["bf16", "f32"])
@pytest.mark.parametrize("rows_gate", [False, True])
@pytest.mark.parametrize("B,H", [(2, 64), (700, 2048), (5, 1002), (3, 9)])
def test_norm_gates_without_a_finite_value(m, res, rows_gate, B, H):  # noqa: F811
    """Gates of +inf, -inf and NaN: all of y, nothing of it, and NaN in that element alone."""
    rt = torch.bfloat16 if res == "bf16" else torch.float32
    h = torch.ones(B, H, dtype=rt, device="cuda")
    y = torch.full((B, H), 2.0, dtype=torch.bfloat16, device="cuda")
    g = torch.zeros(B if rows_gate else 1, H, dtype=torch.bfloat16, device="cuda")
    g[:, 0], g[:, 3], g[:, 8] = float("inf"), -float("inf"), float("nan")
    m.moe_block_norm(h, y, None, g, None, h, None, B, H, res_dtype=m.MOE_T_BF16 if res == "bf16" else m.MOE_T_F32,
                     gate_kind=m.MOE_GATE_SIGMOID, gate_stride=H if rows_gate else 0)
    assert bool(((h[:, 0] - 3.0).abs() <= 8 * U * 3).all()) and bool((h[:, 3] == 1.0).all())
    assert bool(h[:, 8].isnan().all()) and int(h.isnan().sum()) == B
    keep = torch.tensor([i for i in range(H) if i not in (0, 3, 8)], device="cuda")
    assert bool(((h[:, keep] - 2.0).abs() <= 8 * U * 2).all())

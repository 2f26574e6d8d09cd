"""Host side of the operators around the experts: refusals before anything is
enqueued, and the reference's own number formats."""
import numpy as np
import pytest
import torch

from tests import block_ref as ref

P = 0x10000  # an aligned address; the calls below are refused before it is used


@pytest.fixture(scope="module")
def m():
    import __graft_entry__
    __graft_entry__._build_module().build()
    import expert_slot_cache_lru_gb300 as mod
    return mod


def refused(m, code, call):
    with pytest.raises(m.MoeError) as ei:
        call()
    assert ei.value.code == code


def norm(m, **kw):
    a = dict(d_h=P, d_y=P * 2, d_post_w=P * 3, d_gate=None, d_pre_w=P * 5, d_h_out=P * 6,
             d_x_out=P * 7, n_rows=2, hidden=64, stream=0)
    a.update(kw)
    return lambda: m.moe_block_norm(**a)


@pytest.mark.parametrize("kw", [
    dict(n_rows=-1), dict(hidden=0), dict(res_dtype=2), dict(gate_kind=3), dict(d_h=None),
    dict(gate_kind=1), dict(d_gate=P), dict(d_pre_w=None), dict(d_x_out=None), dict(d_y=None),
    dict(d_h_out=None, d_x_out=None, d_pre_w=None), dict(h_stride=63), dict(y_stride=-64),
    dict(d_gate=P, gate_kind=1, gate_stride=8), dict(d_h=P + 1), dict(res_dtype=1, d_h=P + 2),
    dict(d_x_out=P * 7 + 1), dict(d_h_out=P, h_out_stride=128), dict(d_x_out=P), dict(d_h_out=P * 2),
    dict(d_x_out=P * 2, x_out_stride=128), dict(d_h_out=P * 7)])
def test_block_norm_refuses(m, kw):
    refused(m, m.MOE_ERR_INVALID_ARG, norm(m, **kw))


def test_block_norm_limits(m):
    refused(m, m.MOE_ERR_UNSUPPORTED, norm(m, hidden=32769))
    norm(m, n_rows=0)()  # nothing enqueued


def route(m, **kw):
    a = dict(d_x=P, d_router=P * 2, d_bias=None, n_rows=2, hidden=64, n_experts=32, k=4,
             d_logits=P * 3, d_ids=P * 4, d_w=P * 5, stream=0)
    a.update(kw)
    return lambda: m.moe_route(**a)


@pytest.mark.parametrize("kw", [
    dict(n_rows=-1), dict(hidden=0), dict(n_experts=0), dict(k=0), dict(k=33), dict(score=2),
    dict(n_groups=0), dict(n_groups=5), dict(topk_groups=0), dict(topk_groups=2), dict(group_top=3),
    dict(n_groups=32, group_top=2), dict(d_x=None), dict(d_router=None), dict(d_logits=None),
    dict(d_ids=None), dict(d_w=None), dict(x_stride=63), dict(d_x=P + 1), dict(d_logits=P + 2),
    dict(d_ids=P + 1), dict(d_bias=P + 2), dict(d_status=P + 4)])
def test_route_refuses(m, kw):
    refused(m, m.MOE_ERR_INVALID_ARG, route(m, **kw))


def test_route_limits(m):
    refused(m, m.MOE_ERR_UNSUPPORTED, route(m, n_experts=16385))
    refused(m, m.MOE_ERR_UNSUPPORTED, route(m, n_experts=64, k=33))
    refused(m, m.MOE_ERR_UNSUPPORTED, route(m, n_experts=65, n_groups=65))
    route(m, n_rows=0)()


@pytest.mark.parametrize("kw", [dict(dtype=2), dict(d_logits=None), dict(logits_stride=31),
                                dict(d_logits=P + 2), dict(d_ids=None), dict(d_w=P + 2), dict(k=33)])
def test_route_logits_refuses(m, kw):
    a = dict(d_logits=P, dtype=m.MOE_T_F32, d_bias=None, n_rows=2, n_experts=32, k=4, d_ids=P * 4,
             d_w=P * 5, stream=0)
    a.update(kw)
    refused(m, m.MOE_ERR_INVALID_ARG, lambda: m.moe_route_logits(**a))


@pytest.mark.parametrize("kw", [
    dict(wfmt=9), dict(dtype=2), dict(rows=-1), dict(cols=0), dict(cols=40), dict(wfmt=2, cols=48),
    dict(wfmt=2, d_global=P), dict(d_global=P + 2), dict(d_codes=None), dict(d_scales=P + 8),
    dict(d_codes=P + 4)])
def test_fp4_conversions_refuse(m, kw):
    a = dict(wfmt=m.MOE_W_NVFP4, dtype=m.MOE_T_BF16, rows=2, cols=64, d_global=None, d_codes=P,
             d_scales=P * 2, stream=0)
    a.update(kw)
    refused(m, m.MOE_ERR_INVALID_ARG, lambda: m.moe_fp4_quantize(d_src=P * 3, **a))
    refused(m, m.MOE_ERR_INVALID_ARG, lambda: m.moe_fp4_dequantize(d_dst=P * 3, **a))


def test_fp4_conversions_limits(m):
    for fmt in (m.MOE_W_BF16, m.MOE_W_Q4_0):
        refused(m, m.MOE_ERR_UNSUPPORTED,
                lambda: m.moe_fp4_quantize(fmt, P, 0, 2, 64, None, P, P, stream=0))
    for kw in (dict(src_stride=63), dict(d_src=None), dict(d_src=P + 1)):
        a = dict(wfmt=1, d_src=P, dtype=0, rows=2, cols=64, d_global=None, d_codes=P, d_scales=P, stream=0)
        a.update(kw)
        refused(m, m.MOE_ERR_INVALID_ARG, lambda: m.moe_fp4_quantize(**a))
    for kw in (dict(d_global=None), dict(rows=-1), dict(src_stride=63), dict(d_src=P + 2)):
        a = dict(d_src=P, dtype=1, rows=2, cols=64, d_global=P, stream=0)
        a.update(kw)
        refused(m, m.MOE_ERR_INVALID_ARG, lambda: m.moe_fp4_global_scale(**a))
    m.moe_fp4_quantize(1, None, 0, 0, 64, None, None, None, stream=0)


@pytest.mark.parametrize("kw", [
    dict(wfmt=7), dict(n_rows=-1), dict(n=0), dict(k=0), dict(k=48), dict(dtype=5),
    dict(d_x_codes=None), dict(d_w_scales=None), dict(d_w_codes=P + 8), dict(d_x_scales=P + 4),
    dict(d_out=None), dict(d_out=P + 2), dict(out_stride=15), dict(d_xg=P + 1), dict(d_status=P + 4),
    dict(wfmt=2, d_wg=P)])
def test_fp4_linear_refuses(m, kw):
    a = dict(wfmt=1, d_x_codes=P, d_x_scales=P, d_xg=None, d_w_codes=P, d_w_scales=P, d_wg=None,
             n_rows=2, n=16, k=64, d_out=P, dtype=m.MOE_T_F32, stream=0)
    a.update(kw)
    refused(m, m.MOE_ERR_INVALID_ARG, lambda: m.moe_fp4_linear(**a))


def test_fp4_linear_limits(m):
    refused(m, m.MOE_ERR_UNSUPPORTED,
            lambda: m.moe_fp4_linear(3, P, P, None, P, P, None, 2, 16, 64, P, 1, stream=0))
    m.moe_fp4_linear(1, P, P, None, P, P, None, 0, 16, 64, P, 1, stream=0)


def test_reference_formats_agree_with_torch():
    codes = torch.arange(127, dtype=torch.uint8)
    assert np.array_equal(ref.E4M3, codes.view(torch.float8_e4m3fn).double().numpy())
    v = np.random.default_rng(0).uniform(0, 448, 4000).astype(np.float32)
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.nearest(v, ref.E4M3), want)
    ties = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0])
    assert ref.E2M1[ref.nearest(ties, ref.E2M1)].tolist() == [0, 1, 1, 2, 2, 4, 4, 6]


def test_reference_route_by_hand():
    z = np.array([[1.0, 3.0, 3.0, -np.inf], [np.nan, -np.inf, -np.inf, -np.inf]])
    ids, w, _ = ref.route(z, 3)
    assert ids.tolist() == [[1, 2, 0], [-1, -1, -1]]
    e = np.exp([3.0, 3.0, 1.0])
    assert np.allclose(w[0], e / e.sum()) and not w[1].any()
    # groups of two: the best single expert sits in a group whose sum loses
    z = np.array([[4.0, -4.0, 2.0, 2.0]])
    ids, _, _ = ref.route(z, 2, score="sigmoid", bias=np.zeros(4), groups=2, topk_groups=1, group_top=2)
    assert ids.tolist() == [[2, 3]]

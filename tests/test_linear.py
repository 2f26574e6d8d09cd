"""Host side of the bf16 products, the grouping and the combine: refusals before
anything is enqueued, and the reference's own order."""
import numpy as np
import pytest

from tests import linear_ref as ref

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


def linear(m, **kw):
    a = dict(d_x=P, d_w=P * 2, d_bias=P * 3, d_res=P * 4, d_out=P * 5, n_rows=2, n=48, k=64, stream=0)
    a.update(kw)
    return lambda: m.moe_linear(**a)


@pytest.mark.parametrize("kw", [
    dict(n_rows=-1), dict(n=0), dict(k=0), dict(act=-1), dict(act=5), dict(gated=2), dict(dtype=2),
    dict(x_stride=63), dict(w_stride=-64), dict(res_stride=47), dict(out_stride=47), dict(d_x=None),
    dict(d_w=None), dict(d_out=None), dict(d_x=P + 1), dict(d_w=P + 1), dict(d_bias=P + 1),
    dict(d_res=P + 1), dict(d_out=P + 1), dict(dtype=1, d_out=P * 5 + 2), dict(dtype=1, d_res=P * 4 + 2),
    dict(d_status=P + 4), dict(d_res=P * 5, out_stride=64), dict(d_out=P), dict(d_out=P * 2)])
def test_linear_refuses(m, kw):
    refused(m, m.MOE_ERR_INVALID_ARG, linear(m, **kw))


def test_linear_without_rows(m):
    linear(m, n_rows=0)()
    linear(m, n_rows=0, d_x=None, d_w=None, d_out=None)()


def grouped(m, **kw):
    a = dict(d_x=P, x_rows=4, d_order=P * 2, per_row=2, d_offsets=P * 3, n_groups=3, d_w=P * 4,
             d_bias=None, d_out=P * 5, n_rows=8, n=48, k=64, stream=0)
    a.update(kw)
    return lambda: m.moe_grouped_linear(**a)


@pytest.mark.parametrize("kw", [
    dict(n_rows=-1), dict(n=0), dict(k=0), dict(act=7), dict(gated=-1), dict(dtype=3), dict(n_groups=0),
    dict(per_row=0), dict(x_rows=-1), dict(d_order=None), dict(d_offsets=None), dict(d_offsets=P * 3 + 2),
    dict(d_order=P * 2 + 1), dict(w_group_stride=48 * 64 - 1), dict(gated=True, w_group_stride=48 * 64),
    dict(w_stride=72, w_group_stride=48 * 64), dict(x_stride=8), dict(out_stride=40), dict(d_out=P * 4),
    dict(d_x=None), dict(d_bias=P + 1)])
def test_grouped_linear_refuses(m, kw):
    refused(m, m.MOE_ERR_INVALID_ARG, grouped(m, **kw))


def test_grouped_linear_limits(m):
    refused(m, m.MOE_ERR_UNSUPPORTED, grouped(m, n_groups=16385))
    grouped(m, n_rows=0)()
    grouped(m, x_rows=0)()  # no place has a row: nothing enqueued


@pytest.mark.parametrize("kw", [
    dict(n_routes=-1), dict(n_experts=0), dict(d_ids=None), dict(d_offsets=None), dict(d_ids=P + 2),
    dict(d_offsets=P * 2 + 1), dict(d_order=P * 3 + 2), dict(d_pos=P * 4 + 1), dict(d_order=P),
    dict(d_order=P * 4), dict(d_offsets=P), dict(d_offsets=P * 3), dict(d_offsets=P * 4)])
def test_group_routes_refuses(m, kw):
    a = dict(d_ids=P, n_routes=8, n_experts=4, d_offsets=P * 2, d_order=P * 3, d_pos=P * 4, stream=0)
    a.update(kw)
    refused(m, m.MOE_ERR_INVALID_ARG, lambda: m.moe_group_routes(**a))


def test_group_routes_limits(m):
    refused(m, m.MOE_ERR_UNSUPPORTED, lambda: m.moe_group_routes(P, 8, 16385, P * 2, stream=0))


@pytest.mark.parametrize("kw", [
    dict(n_rows=-1), dict(k=0), dict(hidden=0), dict(y_rows=-1), dict(dtype=2), dict(y_dtype=2),
    dict(y_dtype=1), dict(y_stride=63), dict(add_stride=63), dict(out_stride=-1), dict(d_y=None),
    dict(d_pos=None), dict(d_w=None), dict(d_out=None), dict(d_y=P + 1), dict(d_pos=P * 2 + 2),
    dict(d_w=P * 3 + 1), dict(d_add=P * 4 + 1), dict(d_out=P * 5 + 1), dict(dtype=1, d_out=P * 5 + 2),
    dict(d_out=P), dict(d_add=P * 5, out_stride=128)])
def test_combine_refuses(m, kw):
    a = dict(d_y=P, y_rows=8, d_pos=P * 2, d_w=P * 3, d_add=P * 4, d_out=P * 5, n_rows=2, k=4, hidden=64,
             stream=0)
    a.update(kw)
    refused(m, m.MOE_ERR_INVALID_ARG, lambda: m.moe_combine(**a))


def test_combine_without_rows(m):
    m.moe_combine(None, 0, None, None, None, None, 0, 4, 64, stream=0)


def test_the_reference_order():
    offsets, order, pos = ref.group([2, 0, -1, 2, 5, 0], 3)
    assert offsets.tolist() == [0, 2, 2, 4]
    assert order.tolist() == [1, 5, 0, 3, -1, -1]
    assert pos.tolist() == [2, 0, -1, 3, -1, 1]
    assert np.array_equal(ref.group([], 2)[0], [0, 0, 0])

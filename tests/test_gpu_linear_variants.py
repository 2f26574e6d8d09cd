"""Each form of the bf16 products of few rows that the sizes choose, and GELU at arguments that
are no bf16 numbers."""
import pytest
import torch

from tests import linear_ref as ref
from tests.test_gpu_linear import BF16, grouped_case, linear_case, m  # noqa: F401

pytestmark = pytest.mark.gpu

FORMS = [dict(), dict(kind="silu", bias=True, res=True, alpha=0.22, f32=True), dict(kind="gelu", res=True, alias=True)]


# few results with long sums: one and two rows, dot products of 16 warps
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("B,N,K,gated", [(1, 1024, 8192, False), (1, 1, 4096, False), (1, 512, 4096, True),
                                         (1, 77, 8200, True), (2, 1000, 8192, False), (2, 33, 4104, False),
                                         (2, 304, 4096, True), (2, 5, 16384, True)])
def test_few_results_of_one_or_two_rows(m, form, B, N, K, gated):  # noqa: F811
    linear_case(m, B, N, K, gated=gated, **form)


# 3 to 16 rows, 32 warps
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("B,N,K,gated", [(3, 2400, 4096, False), (8, 17, 8192, False), (5, 600, 8192, True),
                                         (8, 9, 4104, True), (9, 1024, 8192, False), (16, 15, 4096, False),
                                         (11, 77, 4096, True), (16, 512, 8184, True)])
def test_few_results_of_three_to_sixteen_rows(m, form, B, N, K, gated):  # noqa: F811
    linear_case(m, B, N, K, gated=gated, **form)


# tiles of 32, of 128, of a pair's 128 and 256 tokens, K in one, two and four parts, one and several tiles a CTA
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("B,N,K", [(20, 64, 1280), (40, 2500, 2048), (20, 64, 2048), (2000, 300, 1280), (40, 2500, 8192),
                                   (40, 12000, 1280), (300, 12000, 1280), (40, 8192, 8192), (100, 12000, 1280),
                                   (2000, 2500, 1280), (300, 4096, 16384)])
def test_tiles_and_parts(m, form, B, N, K):  # noqa: F811
    linear_case(m, B, N, K, **form)


# more groups than four times the places: 17 to 48 of them one by one, and the sizes next to these
@pytest.mark.parametrize("kw", [dict(kind="silu", gated=True), dict(bias=True, f32=True), dict(gather=False),
                                dict(bad=3, top=8)])
@pytest.mark.parametrize("places,E", [(17, 68), (17, 67), (20, 256), (32, 128), (48, 192), (48, 300), (49, 300)])
def test_places_of_many_groups(m, kw, places, E):  # noqa: F811
    counts = [0] * E
    for p in range(places):  # mostly apart, some groups with two, the first and the last among them
        counts[(p if p % 5 else p // 2) * (E - 1) // (places - 1)] += 1
    for N, K in ((96, 256), (64, 4096)):
        grouped_case(m, counts, N, K, spare=0, **kw)
    grouped_case(m, counts[:-1] + [counts[-1] - 1], 96, 256, spare=1, **kw)


# more places than groups, either side of what the matrices read again may amount to
@pytest.mark.parametrize("kw", [dict(kind="silu", gated=True, bias=True), dict(f32=True), dict(gather=False)])
@pytest.mark.parametrize("counts,N,K", [([16], 1024, 2176), ([16], 1024, 2240), ([0, 7, 0, 9], 1200, 2048),
                                        ([1, 1, 1, 0], 4096, 4096), ([2], 4096, 8192), ([2], 4104, 8192),
                                        ([3, 2], 2048, 4096), ([1], 8192, 8192)])
def test_more_places_than_groups(m, kw, counts, N, K):  # noqa: F811
    grouped_case(m, counts, N // 2 if kw.get("gated") else N, K, spare=0, **kw)


@pytest.mark.parametrize("rows", [1, 3, 20])
def test_gelu_of_fp32_arguments(m, rows):  # noqa: F811
    """z is any fp32 number: three bf16 weights of which each holds what the ones before leave, times one.  They are
    one lane's or one addition's products, no more than 24 bits together: z is exact."""
    g = torch.Generator().manual_seed(3)
    z = torch.cat([torch.rand(300000, generator=g) * 6 - 3, torch.rand(300000, generator=g) * 30 - 15,
                   torch.rand(100000, generator=g) * 0.01 - 0.005]).cuda()
    N, K = z.numel(), 8
    w = torch.zeros(N, K, dtype=BF16, device="cuda")
    left = z.clone()
    for j in range(3):
        w[:, j] = (left.view(torch.int32) & -65536).view(torch.float32).to(BF16)  # the upper half of its bits
        left -= w[:, j].float()
    assert (left == 0).all() and (w.double().sum(1) == z.double()).all()
    x = torch.ones(rows, K, dtype=BF16, device="cuda")
    plain, out = (torch.empty(rows, N, device="cuda") for _ in range(2))
    m.moe_linear(x, w, None, None, plain, rows, N, K, dtype=m.MOE_T_F32)
    m.moe_linear(x, w, None, None, out, rows, N, K, act=m.MOE_ACT_GELU, dtype=m.MOE_T_F32)
    assert (plain == z).all()
    y, e = ref.act(z.double(), "gelu")
    assert ((out.double() - y).abs() <= e).all()

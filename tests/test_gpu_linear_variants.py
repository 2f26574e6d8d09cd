"""Each form of the bf16 products of few rows that the sizes choose."""
import pytest

from tests.test_gpu_linear import grouped_case, linear_case, m  # noqa: F401

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

"""fp32 results of the bf16 products over long sums: no error that grows with K as one chain of
the tensor cores' truncated additions does, whichever kernel takes the call."""
import numpy as np
import pytest
import torch

from tests.test_gpu_linear import BF16, gen, linear_case, m, normal, padded  # noqa: F401

pytestmark = pytest.mark.gpu


def sum_bound(K):
    """Off by, relative to the norm of the results.  A chain takes 16 products an addition, at most 256 of K:
    16 additions, each truncated, by at most 2^-23 of the running sum, half of that on average, always the same
    way.  A sum of random products grows with the root of its length, so the running sum is two thirds of the
    chain's on average.  Chains are independent of one another: their errors grow with the root of their number,
    as the whole sum does, so K does not enter.  They (as sums of 16 products, where these are chains) are added
    in fp32, rounded to nearest: an error spread evenly over half of 2^-23 of the running sum either way,
    2^-24 / sqrt 3 on average, at random signs; the running sum's square is half of the whole's on average:
    sqrt(n / 6) 2^-24 for n.
    Chains of 512 would be off by up to twice the first term, one of 4,096 by sixteen times."""
    return 256 / 16 * 2 / 3 * 2.0 ** -24 + (K / 16 / 6) ** 0.5 * 2.0 ** -24


def off_by(out, y):
    return ((out.double() - y).norm() / y.norm()).item()


def dense(m, B, N, K, gated=False, pad=0, off=0):  # noqa: F811
    g = gen(B, N, K, gated)
    x = padded(normal(g, B, K), pad, off)
    w = padded(normal(g, N * (1 + gated), K, std=K ** -0.5), pad, off)
    outs = [torch.full((B, N), float("nan"), device="cuda") for _ in range(2)]
    st = torch.zeros(1, dtype=torch.int64, device="cuda")
    for out in outs:
        m.moe_linear(x, w, None, None, out, B, N, K, gated=gated, dtype=m.MOE_T_F32, x_stride=K + pad,
                     w_stride=K + pad, d_status=st)
    z = x.double() @ w.double().T
    y = z[:, :N] * z[:, N:] if gated else z
    assert st.item() == 0
    # a gated result is a product of two sums
    assert off_by(outs[0], y) < sum_bound(K) * (1 + gated)
    assert torch.equal(*outs)


# tiles of 32, 128 and a pair's 128 tokens; K cut over clusters and not; one and several tiles a CTA; widths that end
# inside one
@pytest.mark.parametrize("B,N,K", [(20, 128, 16384), (30, 4096, 16384), (64, 512, 65536), (100, 20000, 2048),
                                   (300, 300, 16384), (300, 1024, 4096), (1000, 5000, 1280), (1000, 5000, 1344),
                                   (2000, 2500, 2048), (2000, 2500, 2056), (3000, 4096, 16384), (5000, 2056, 8192),
                                   (20, 8192, 2112), (2000, 64, 8192), (2000, 300, 1280), (40, 2500, 8192),
                                   (500, 1024, 16384), (40, 12000, 1280), (200, 12000, 1280), (40, 8192, 8192)])
def test_long_sums(m, B, N, K):  # noqa: F811
    dense(m, B, N, K)


@pytest.mark.parametrize("B,N,K", [(30, 512, 16384), (200, 96, 8192), (1500, 1024, 4096), (1500, 1024, 16384),
                                   (40, 2048, 8192), (40, 4096, 8192)])
def test_long_sums_gated(m, B, N, K):  # noqa: F811
    dense(m, B, N, K, gated=True)


@pytest.mark.parametrize("B,N,K,gated", [(300, 300, 131072, False), (300, 300, 65600, True), (20, 128, 1 << 21, False)])
def test_the_longest_sums_of_bf16_results(m, B, N, K, gated):  # noqa: F811
    linear_case(m, B, N, K, gated=gated, kind="silu" if gated else "none", bias=True, res=True)


# rows that are no whole 16-byte pieces; gated widths that are no multiple of 16
@pytest.mark.parametrize("B,N,K,gated,pad,off", [
    (17, 40, 4097, False, 0, 0), (200, 300, 4097, False, 0, 0), (200, 300, 8191, False, 0, 0),
    (150, 130, 16384, False, 1, 0), (150, 130, 16384, False, 0, 1), (300, 100, 4097, True, 0, 0),
    (300, 1000, 4096, True, 0, 0), (40, 33, 32768, True, 0, 0)])
def test_long_sums_of_any_layout(m, B, N, K, gated, pad, off):  # noqa: F811
    dense(m, B, N, K, gated, pad, off)


# few rows, whole and not
@pytest.mark.parametrize("B", [1, 2, 5, 16])
@pytest.mark.parametrize("N,K,pad", [(64, 4096, 0), (300, 8192, 0), (64, 65536, 0), (64, 8191, 0), (48, 65536, 1)])
def test_long_sums_of_few_rows(m, B, N, K, pad):  # noqa: F811
    dense(m, B, N, K, pad=pad)


@pytest.mark.parametrize("E,mean,N,K,gated,gather", [
    (6, 30, 512, 16384, False, True), (3, 700, 520, 16384, False, False), (40, 300, 1024, 4096, False, True),
    (40, 300, 1024, 2048, True, True), (64, 40, 1024, 1344, False, False), (100, 150, 512, 8192, False, True),
    (6, 30, 100, 4097, False, True), (6, 90, 100, 8191, False, False), (5, 60, 200, 4096, True, True),
    (8, 1, 128, 32768, False, True)])
def test_long_sums_in_groups(m, E, mean, N, K, gated, gather):  # noqa: F811
    r = np.random.default_rng([E, mean, K])
    ends = np.concatenate(([0], np.cumsum(r.poisson(mean, E))))
    rows = int(ends[-1])
    g = gen(E, mean, N, K)
    offsets = torch.tensor(ends, dtype=torch.int32, device="cuda")
    x, w = normal(g, rows, K), normal(g, E, N * (1 + gated), K, std=K ** -0.5)
    order = torch.randperm(rows, generator=g, device="cuda").int() if gather else None
    out = torch.full((rows, N), float("nan"), device="cuda")
    m.moe_grouped_linear(x, rows, order, 1, offsets, E, w, None, out, rows, N, K, gated=gated, dtype=m.MOE_T_F32)
    src = x[order.long()] if gather else x
    z = torch.cat([src[a:b].double() @ w[e].double().T for e, (a, b) in enumerate(zip(ends[:-1], ends[1:]))])
    y = z[:, :N] * z[:, N:] if gated else z
    assert off_by(out, y) < sum_bound(K) * (1 + gated)


@pytest.mark.parametrize("E,mean,N,K,gated,gather", [(300, 2, 512, 2048, True, True), (40, 60, 520, 4096, False, False),
                                                     (30, 90, 256, 1344, True, True)])
def test_bf16_results_of_short_groups(m, E, mean, N, K, gated, gather):  # noqa: F811
    """The sums of fp32 results, rounded: the same chains whatever the type."""
    r = np.random.default_rng([E, mean, K])
    ends = np.concatenate(([0], np.cumsum(r.poisson(mean, E))))
    rows = int(ends[-1])
    assert 48 < rows < 100 * E
    g = gen(E, mean, N, K)
    offsets = torch.tensor(ends, dtype=torch.int32, device="cuda")
    x, w = normal(g, rows, K), normal(g, E, N * (1 + gated), K, std=K ** -0.5)
    order = torch.randperm(rows, generator=g, device="cuda").int() if gather else None
    wide, out = (torch.full((rows, N), float("nan"), dtype=t, device="cuda") for t in (torch.float32, BF16))
    for o, t in ((wide, m.MOE_T_F32), (out, m.MOE_T_BF16)):
        m.moe_grouped_linear(x, rows, order, 1, offsets, E, w, None, o, rows, N, K, act=m.MOE_ACT_SILU, gated=gated,
                             dtype=t)
    assert torch.equal(out, wide.to(BF16))


def test_long_sums_captured_on_two_streams(m):  # noqa: F811
    """Graphs of dense products, cut over clusters and not, and of groups, replayed at once and again."""
    def calls(side):
        g = gen("two", side)
        offsets = torch.tensor([0, 40, 40, 300, 411], dtype=torch.int32, device="cuda")
        some = [(normal(g, B, K), normal(g, N, K, std=K ** -0.5)) for B, N, K in ((40, 2500, 8192), (700, 1000, 4096))]
        x, w = normal(g, 411, 4096), normal(g, 4, 256, 4096, std=1 / 64)
        outs = [torch.empty(a.shape[0], b.shape[0], device="cuda") for a, b in (*some, (x, w[0]))]

        def go():
            for (a, b), o in zip(some, outs):
                m.moe_linear(a, b, None, None, o, a.shape[0], b.shape[0], a.shape[1], dtype=m.MOE_T_F32)
            m.moe_grouped_linear(x, 411, None, 1, offsets, 4, w, None, outs[2], 411, 256, 4096, dtype=m.MOE_T_F32)

        go()
        torch.cuda.synchronize()
        want = [o.clone() for o in outs]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            go()
            go()
        return graph, outs, want, (some, offsets, x, w)  # the graph's inputs live as long as it

    sides = [calls(i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in sides]
    for _, outs, _, _ in sides:
        for o in outs:
            o.fill_(float("nan"))
    torch.cuda.synchronize()
    for _ in range(5):
        for (graph, *_), s in zip(sides, streams):
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for _, outs, want, _ in sides:
        assert all(torch.equal(o, a) for o, a in zip(outs, want))

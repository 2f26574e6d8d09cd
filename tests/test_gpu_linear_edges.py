"""The bf16 products, the grouping and the combine where they are largest, on several
streams, and after a wait has run out: the tensor-core kernel is built once more with a limit
of a few cycles on its waits, so that a CTA gives up at the first copy or further on; it reports
it, its copies land, and what it stored is right or untouched."""
import ctypes as C
import os
import subprocess

import numpy as np
import pytest
import torch

from tests import linear_ref as ref
from tests.test_gpu_linear import BF16, chain, gen, grouped_case, linear_case, m, normal  # noqa: F401

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "expert_slot_cache_lru_gb300", "csrc")

SHIM = r"""
#include "linear.cuh"
extern "C" __attribute__((visibility("default"))) int product(
    const void* x, const void* w, void* out, const int* order, const int* offsets, int x_rows, int per_row,
    int groups, int rows, int n, int k, int gated, int sms, unsigned long long* status, void* stream) {
  moe::Linear l{};
  l.x = static_cast<const __nv_bfloat16*>(x), l.w = static_cast<const __nv_bfloat16*>(w), l.out = out;
  l.x_stride = l.w_stride = k, l.out_stride = l.res_stride = n, l.group_stride = (long long)n * k * (1 + gated);
  l.order = order, l.offsets = offsets, l.x_rows = x_rows, l.per_row = per_row, l.groups = groups;
  l.rows = rows, l.n = n, l.k = k, l.gated = gated != 0, l.f32 = true, l.alpha = 1.f, l.status = status;
  moe::lin::division_of(per_row, l.per_mul, l.per_shift);
  return (int)moe::launch_linear_tc(l, sms, static_cast<cudaStream_t>(stream));
}
"""


def build(d, name, *flags):
    """The tensor-core kernel by itself, whatever rows the library gives it."""
    shim, lib = str(d / "shim.cu"), str(d / f"lib{name}.so")
    with open(shim, "w") as f:
        f.write(SHIM)
    subprocess.run([os.environ.get("NVCC", "nvcc"), "-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-std=c++17",
                    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden", "-shared", "--threads", "0", *flags,
                    "-I", CSRC, shim, os.path.join(CSRC, "linear_tc.cu"), os.path.join(CSRC, "tc_host.cu"), "-o", lib],
                   check=True)
    lib = C.CDLL(lib)
    lib.product.argtypes = [C.c_void_p] * 5 + [C.c_int] * 8 + [C.c_void_p] * 2
    return lib


@pytest.fixture(scope="module")
def patient(tmp_path_factory):
    return build(tmp_path_factory.mktemp("patient"), "patient")


@pytest.fixture(scope="module", params=[0, 4000, 12000])
def impatient(request, tmp_path_factory):
    lib = build(tmp_path_factory.mktemp("impatient"), "impatient", f"-DMOE_TC_WAIT_CYCLES={request.param}")
    lib.cycles = request.param
    return lib


def give_up(lib, patient, out, run, what):
    """run(library, status): one product into out."""
    def full():
        st = torch.zeros(1, dtype=torch.int64, device="cuda")
        out.fill_(float("nan"))
        assert run(patient, st) == 0 and st.item() == 0
        return out

    want = full().clone()
    again = full().clone()
    keep = want.isnan()                       # no place of a group
    assert torch.equal(want[~keep], again[~keep]) and torch.equal(keep, again.isnan())
    gave_up = 0
    for _ in range(3):
        out.fill_(float("nan"))
        st = torch.zeros(1, dtype=torch.int64, device="cuda")
        assert run(lib, st) == 0
        torch.cuda.synchronize()              # the context is as it was
        untouched = out.isnan()
        assert torch.equal(out[~untouched], want[~untouched]) and untouched[keep].all()
        assert st.item() == 4 if (untouched & ~keep).any() else st.item() in (0, 4)
        gave_up += int(st.item() != 0)
    if lib.cycles == 0:
        assert gave_up                        # the first copy takes longer
    after = full()
    assert torch.equal(after[~keep], want[~keep])   # tensor memory and barriers were left as they should be
    print(f"{what}: {gave_up} of 3 gave up")


# one CTA a tile, K in two and four parts, tiles of 128, pairs, one and several tiles a CTA
@pytest.mark.parametrize("B,N,K,gated", [(16, 128, 256, 0), (16, 4096, 4096, 0), (30, 512, 2048, 1), (64, 4096, 4096, 0),
                                         (600, 768, 2048, 1), (512, 2048, 2048, 0), (700, 20000, 512, 0),
                                         (2048, 8192, 1024, 0), (3000, 4096, 2048, 1),
                                         (2000, 128, 1024, 0)])
def test_a_wait_that_runs_out(impatient, patient, B, N, K, gated):
    g = gen(B, N, K)
    x, w = normal(g, B, K), normal(g, N * (1 + gated), K, std=K ** -0.5)
    out = torch.empty(B, N, device="cuda")
    sms = torch.cuda.get_device_properties(0).multi_processor_count

    def run(lib, st):
        return lib.product(x.data_ptr(), w.data_ptr(), out.data_ptr(), None, None, B, 1, 1, B, N, K, gated, sms,
                           st.data_ptr(), torch.cuda.current_stream().cuda_stream)

    give_up(impatient, patient, out, run, f"{B} x {N} x {K}")
    y, dy = ref.product(x, w, None, "none", bool(gated), chain(K, True))
    ref.check(out, y, dy, torch.float32)


@pytest.mark.parametrize("E,mean,N,K,gated", [(64, 4, 256, 512, 1), (300, 2, 512, 1024, 0), (16, 300, 512, 1024, 1),
                                              (40, 90, 1000, 2048, 0)])
@pytest.mark.parametrize("gather", [True, False])
def test_a_wait_of_the_groups_that_runs_out(impatient, patient, E, mean, N, K, gated, gather):
    r = np.random.default_rng([E, mean])
    counts = r.poisson(mean, E)
    placed = int(counts.sum())
    rows, per = placed + 5, 3
    g = gen(E, mean, N)
    offsets = torch.tensor(np.concatenate(([0], np.cumsum(counts))), dtype=torch.int32, device="cuda")
    x = normal(g, rows, K)
    order = torch.randint(0, rows * per, (rows,), generator=g, device="cuda").int() if gather else None
    w = normal(g, E, N * (1 + gated), K, std=K ** -0.5)
    out = torch.empty(rows, N, device="cuda")
    sms = torch.cuda.get_device_properties(0).multi_processor_count

    def run(lib, st):
        return lib.product(x.data_ptr(), w.data_ptr(), out.data_ptr(), order.data_ptr() if gather else None,
                           offsets.data_ptr(), rows, per, E, rows, N, K, gated, sms, st.data_ptr(),
                           torch.cuda.current_stream().cuda_stream)

    give_up(impatient, patient, out, run, f"{E} groups of {mean}")


@pytest.mark.parametrize("per_row", [1, 3, 7, 8, 1000])
def test_places_of_any_number_a_row(m, per_row):  # noqa: F811
    grouped_case(m, [5, 0, 40, 17], 64, 128, top=per_row, gated=True, kind="silu")
    grouped_case(m, [300, 2], 96, 72, top=per_row)


@pytest.mark.parametrize("K", [64, 128, 192, 256, 320, 384])
def test_short_sums_in_parts(m, K):  # noqa: F811
    """Few rows and few tiles: K would be cut into more parts than it has stages."""
    for B in (5, 16, 32, 64, 100):
        linear_case(m, B, 128, K, bias=True)
        linear_case(m, B, 64, K, gated=True, kind="silu")


def test_offsets_that_go_back(m):  # noqa: F811
    """Offsets no grouping writes, many groups: nothing outside the rows is touched and the call ends."""
    g = gen(9)
    N, K, rows, E = 128, 64, 3000, 600
    x, w = normal(g, rows, K), normal(g, E, N, K)
    big = torch.full((rows + 512, N), -7.0, dtype=BF16, device="cuda")
    out = big[256:256 + rows]
    r = np.random.default_rng(3)
    for offs in ([0, rows] * ((E + 1) // 2 + 1), r.integers(-10 ** 9, 10 ** 9, E + 1), r.integers(-50, rows + 50, E + 1),
                 [rows] * (E + 1), [2 ** 31 - 1, -2 ** 31] * (E // 2 + 1)):
        o = torch.tensor(np.asarray(offs[:E + 1]), dtype=torch.int64, device="cuda").int()
        for order in (None, torch.arange(rows, device="cuda").int()):
            m.moe_grouped_linear(x, rows, order, 1, o, E, w, None, out, rows, N, K)
            torch.cuda.synchronize()
            assert (big[:256] == -7).all() and (big[256 + rows:] == -7).all()


# ------------------------------------------------------------------ past 32 bits

def test_products_past_32_bits_of_x(m):  # noqa: F811
    B, K, N = 300000, 8192, 16
    x = torch.empty(B, K, dtype=BF16, device="cuda")
    x.normal_(generator=gen(1))
    w = normal(gen(2), N, K, std=K ** -0.5)
    out = torch.empty(B, N, dtype=BF16, device="cuda")
    m.moe_linear(x, w, None, None, out, B, N, K)
    for rows in (slice(0, 64), slice(262100, 262200), slice(B - 70, B)):
        y, dy = ref.product(x[rows], w, None, "none", False, chain(K, True))
        ref.check(out[rows], y, dy, BF16)
    # by an order that names the last rows
    order = torch.arange(B - 1, B - 301, -1, device="cuda").int()
    off = torch.tensor([0, 0, 300], dtype=torch.int32, device="cuda")
    got = torch.empty(300, N, dtype=BF16, device="cuda")
    m.moe_grouped_linear(x, B, order, 1, off, 2, torch.stack([w, w]), None, got, 300, N, K)
    y, dy = ref.product(x[order.long()], w, None, "none", False, chain(K, True))
    ref.check(got, y, dy, BF16)


@pytest.mark.parametrize("N", [131072, 131071])
def test_products_past_32_bits_of_out(m, N):  # noqa: F811
    B, K = 20000, 64
    x, w = normal(gen(1), B, K), normal(gen(2), N, K)
    res = torch.zeros(B, N, dtype=BF16, device="cuda")
    m.moe_linear(x, w, None, res, res, B, N, K)
    for rows in (slice(0, 3), slice(16380, 16390), slice(B - 5, B)):
        y, dy = ref.product(x[rows], w, None, "none", False, chain(K, True))
        ref.check(res[rows], y, dy, BF16)


@pytest.mark.parametrize("rows", [7, 200, 3000])
def test_groups_past_32_bits_of_weights(m, rows):  # noqa: F811
    E, N, K = 1100, 2048, 1024
    w = torch.empty(E, N, K, dtype=BF16, device="cuda")
    w.normal_(generator=gen(3))
    x = normal(gen(4), rows, K)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[1025:] = rows // 2
    off[-1] = rows
    out = torch.empty(rows, N, dtype=BF16, device="cuda")
    m.moe_grouped_linear(x, rows, None, 1, off, E, w, None, out, rows, N, K)
    for part, e in ((slice(0, rows // 2), 1024), (slice(rows // 2, rows), E - 1)):
        y, dy = ref.product(x[part], w[e], None, "none", False, chain(K, True))
        ref.check(out[part], y, dy, BF16)


def test_combine_past_32_bits(m):  # noqa: F811
    P, H, B, k = 600000, 4096, 300000, 2
    y = torch.empty(P, H, dtype=BF16, device="cuda")
    y.normal_(generator=gen(5))
    pos = torch.arange(P - 1, -1, -1, device="cuda").int().view(B, k)
    w = torch.full((B, k), 0.5, device="cuda")
    out = torch.empty(B, H, dtype=BF16, device="cuda")
    m.moe_combine(y, P, pos, w, None, out, B, k, H)
    for rows in (slice(0, 20), slice(262143, 262160), slice(B - 20, B)):
        want = (y[pos[rows].long()].double() * 0.5).sum(1)
        assert ((out[rows].double() - want).abs() <= 2.0 ** -8 * want.abs() * 1.01 + 2.0 ** -20).all()


# ------------------------------------------------------------------ streams

def test_two_streams_at_once(m):  # noqa: F811
    """No state between calls: the same shapes on two streams, many times, give what each gives alone."""
    g = gen(6)
    B, k, E, H, I = 300, 4, 32, 512, 256  # noqa: E741
    w, down = normal(g, E, 2 * I, H, std=H ** -0.5), normal(g, E, H, I, std=I ** -0.5)

    class Side:
        def __init__(self):
            self.s = torch.cuda.Stream()
            self.x = normal(g, B, H)
            self.ids = torch.randint(-1, E, (B, k), generator=g, device="cuda").int()
            self.wt = torch.rand(B, k, generator=g, device="cuda")
            i32 = dict(dtype=torch.int32, device="cuda")
            self.off, self.order, self.pos = torch.empty(E + 1, **i32), torch.empty(B * k, **i32), torch.empty(B * k, **i32)
            self.h, self.y = (torch.zeros(B * k, n, dtype=BF16, device="cuda") for n in (I, H))
            self.out = torch.empty(B, H, dtype=BF16, device="cuda")
            self.d = torch.empty(B, H, dtype=BF16, device="cuda")

        def step(self):
            s = self.s
            m.moe_group_routes(self.ids, B * k, E, self.off, self.order, self.pos, stream=s)
            m.moe_grouped_linear(self.x, B, self.order, k, self.off, E, w, None, self.h, B * k, I, H, act=1, gated=True,
                                 stream=s)
            m.moe_grouped_linear(self.h, B * k, None, 1, self.off, E, down, None, self.y, B * k, H, I, stream=s)
            m.moe_linear(self.x, w[0], None, self.x, self.d, B, H, H, stream=s)
            m.moe_combine(self.y, B * k, self.pos, self.wt, self.d, self.out, B, k, H, stream=s)

    sides = [Side(), Side()]
    torch.cuda.synchronize()
    alone = []
    for a in sides:
        a.step()
        torch.cuda.synchronize()
        alone.append(a.out.clone())
    for _ in range(30):
        for a in sides:
            a.step()
    torch.cuda.synchronize()
    assert all(torch.equal(a.out, b) for a, b in zip(sides, alone))


@pytest.mark.parametrize("R,E", [(8, 256), (900, 2000), (9000, 256), (70000, 256), (70000, 16384)])
def test_order_captured(m, R, E):  # noqa: F811
    """Every cluster size inside a graph, with ids that change between replays."""
    ids = torch.empty(R, dtype=torch.int32, device="cuda")
    off = torch.empty(E + 1, dtype=torch.int32, device="cuda")
    order, pos = torch.empty_like(ids), torch.empty_like(ids)
    graph = torch.cuda.CUDAGraph()
    ids.fill_(-1)
    m.moe_group_routes(ids, R, E, off, order, pos)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        m.moe_group_routes(ids, R, E, off, order, pos)
    for turn in range(3):
        new = np.random.default_rng([R, turn]).integers(-1, E, R).astype(np.int32)
        ids.copy_(torch.from_numpy(new))
        graph.replay()
        torch.cuda.synchronize()
        want = ref.group(new, E)
        for got, w in zip((off, order, pos), want):
            assert np.array_equal(got.cpu().numpy(), w)


def test_captured_on_two_streams(m):  # noqa: F811
    """Two graphs of the same calls, replayed at once."""
    g = gen(7)
    B, N, K = 40, 1024, 1024
    w = normal(g, N, K, std=K ** -0.5)
    x = [normal(g, B, K) for _ in range(2)]
    out = [torch.empty(B, N, dtype=BF16, device="cuda") for _ in range(2)]
    m.moe_linear(x[0], w, None, None, out[0], B, N, K)
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            for _ in range(4):
                m.moe_linear(x[i], w, None, None, out[i], B, N, K)
        graphs.append(gr)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(10):
        for gr, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                gr.replay()
    torch.cuda.synchronize()
    for i in range(2):
        y, dy = ref.product(x[i], w, None, "none", False, chain(K, True))
        ref.check(out[i], y, dy, BF16)


# fp32 results of long sums: K in four parts or more, whatever the tile.  A part has K / 64 additions of 16 products
# or fewer, each truncated: at most 2^-23 of the running sum, half of that on average, and always the same way.  A sum
# of random products grows with the root of its length, so the running sum is two thirds of the whole on average.
# One chain of K / 16 additions would be off by up to four times this (4.4e-6 as measured at K 4,096, beyond the bound).
def long_sum_bound(K):
    return K / 64 * 2 / 3 * 2.0 ** -24


@pytest.mark.parametrize("B,N,K", [(40, 700, 4096), (300, 1024, 4096), (1024, 1024, 4096), (3000, 2048, 4096),
                                   (5000, 2056, 8192)])
def test_fp32_results_of_long_sums(m, B, N, K):
    g = gen(B, N, K)
    x, w = normal(g, B, K), normal(g, N, K, std=K ** -0.5)
    out = torch.empty(B, N, device="cuda")
    m.moe_linear(x, w, None, None, out, B, N, K, dtype=m.MOE_T_F32)
    y = x.double() @ w.double().T
    assert ((out.double() - y).norm() / y.norm()).item() < long_sum_bound(K)
    again = torch.empty_like(out)
    m.moe_linear(x, w, None, None, again, B, N, K, dtype=m.MOE_T_F32)
    assert torch.equal(out, again)


@pytest.mark.parametrize("E,mean,N,K", [(6, 30, 512, 4096), (3, 700, 520, 4096), (40, 300, 1024, 4096)])
def test_fp32_results_of_long_sums_in_groups(m, E, mean, N, K):
    r = np.random.default_rng([E, mean, K])
    ends = np.concatenate(([0], np.cumsum(r.poisson(mean, E))))
    rows = int(ends[-1])
    g = gen(E, mean, N, K)
    offsets = torch.tensor(ends, dtype=torch.int32, device="cuda")
    x, w = normal(g, rows, K), normal(g, E, N, K, std=K ** -0.5)
    out = torch.empty(rows, N, device="cuda")
    m.moe_grouped_linear(x, rows, None, 1, offsets, E, w, None, out, rows, N, K, dtype=m.MOE_T_F32)
    y = torch.cat([x[a:b].double() @ w[e].double().T for e, (a, b) in enumerate(zip(ends[:-1], ends[1:]))])
    assert ((out.double() - y).norm() / y.norm()).item() < long_sum_bound(K)

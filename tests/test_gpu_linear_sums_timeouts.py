"""Long sums of fp32 results after a wait has run out: among the chains that fill the accumulators in turn
nothing half summed is stored."""
from concurrent.futures import ThreadPoolExecutor

import numpy as np
import pytest
import torch

from tests import linear_ref as ref
from tests.test_gpu_linear import chain, gen, normal
from tests.test_gpu_linear_edges import build, give_up

pytestmark = pytest.mark.gpu
LIMITS = (0, 1500, 3000)


@pytest.fixture(scope="module")
def libs(tmp_path_factory):
    """The kernel with its own limit on waits (None) and with those of a few cycles."""
    top = tmp_path_factory.mktemp("long")

    def one(c):
        d = top / str(c)
        d.mkdir()
        lib = build(d, "long", *([] if c is None else [f"-DMOE_TC_WAIT_CYCLES={c}"]))
        lib.cycles = c
        return lib

    with ThreadPoolExecutor(4) as ex:
        return dict(zip((None, *LIMITS), ex.map(one, (None, *LIMITS))))


# tiles of 32, 128 and a pair's 128 tokens; K cut over clusters and not
@pytest.mark.parametrize("cycles", LIMITS)
@pytest.mark.parametrize("B,N,K,gated", [(20, 64, 16384, 0), (300, 1024, 4096, 0), (40, 2500, 8192, 0),
                                         (2000, 300, 1280, 0), (40, 8192, 8192, 0), (200, 12000, 2048, 0),
                                         (1500, 1024, 4096, 1)])
def test_a_wait_that_runs_out(libs, cycles, B, N, K, gated):
    g = gen(B, N, K)
    x, w = normal(g, B, K), normal(g, N * (1 + gated), K, std=K ** -0.5)
    out = torch.empty(B, N, device="cuda")
    sms = torch.cuda.get_device_properties(0).multi_processor_count

    def run(lib, st):
        return lib.product(x.data_ptr(), w.data_ptr(), out.data_ptr(), None, None, B, 1, 1, B, N, K, gated, sms,
                           st.data_ptr(), torch.cuda.current_stream().cuda_stream)

    give_up(libs[cycles], libs[None], out, run, f"{B} x {N} x {K}")
    y, dy = ref.product(x, w, None, "none", bool(gated), chain(K, True))
    ref.check(out, y, dy, torch.float32)


@pytest.mark.parametrize("cycles", LIMITS)
@pytest.mark.parametrize("gather", [True, False])
def test_a_wait_of_the_groups_that_runs_out(libs, cycles, gather):
    E, N, K, per = 16, 512, 4096, 3
    counts = np.random.default_rng(4).poisson(150, E)
    rows = int(counts.sum()) + 5
    g = gen(E, N, K)
    offsets = torch.tensor(np.concatenate(([0], np.cumsum(counts))), dtype=torch.int32, device="cuda")
    x = normal(g, rows, K)
    order = torch.randint(0, rows * per, (rows,), generator=g, device="cuda").int() if gather else None
    w = normal(g, E, N, K, std=K ** -0.5)
    out = torch.empty(rows, N, device="cuda")
    sms = torch.cuda.get_device_properties(0).multi_processor_count

    def run(lib, st):
        return lib.product(x.data_ptr(), w.data_ptr(), out.data_ptr(), order.data_ptr() if gather else None,
                           offsets.data_ptr(), rows, per, E, rows, N, K, 0, sms, st.data_ptr(),
                           torch.cuda.current_stream().cuda_stream)

    give_up(libs[cycles], libs[None], out, run, f"{E} groups")

"""What the tensor-core products do after a wait has run out.  The kernels are built
once more with a limit of a few cycles on every wait but those for copies and MMAs in
flight, so that a wait gives up at the first copy or further on: the CTA reports it,
its copies land, and what it stored is right or untouched."""
import ctypes as C
import os
import subprocess

import numpy as np
import pytest
import torch

from tests import block_ref as ref
from tests.test_gpu_block_ops import U, dev, m  # noqa: F401  (m: the library)

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "expert_slot_cache_lru_gb300", "csrc")

SHIM = r"""
#include "block_ops.cuh"
extern "C" __attribute__((visibility("default"))) int product(
    int nv, const uint8_t* xc, const uint8_t* xs, const uint8_t* wc, const uint8_t* ws, int rows, int n, int k,
    float* out, unsigned long long* status, void* stream) {
  moe::Fp4Linear a{};
  a.xc = xc, a.xs = xs, a.wc = wc, a.ws = ws, a.out = out, a.out_stride = n;
  a.rows = rows, a.n = n, a.k = k, a.nv = nv != 0, a.f32 = true, a.status = status;
  return (int)moe::launch_fp4_linear(a, static_cast<cudaStream_t>(stream));
}
extern "C" __attribute__((visibility("default"))) int logits(const void* x, const void* router, int rows, int hidden,
                                                             int experts, float* z, unsigned long long* status,
                                                             void* stream) {
  return (int)moe::launch_route_logits(static_cast<const __nv_bfloat16*>(x), hidden,
                                       static_cast<const __nv_bfloat16*>(router), rows, hidden, experts, z, status,
                                       static_cast<cudaStream_t>(stream));
}
"""


@pytest.fixture(scope="module", params=[0, 4000, 12000])
def impatient(request, tmp_path_factory):
    d = tmp_path_factory.mktemp("impatient")
    shim, lib = str(d / "shim.cu"), str(d / "libimpatient.so")
    with open(shim, "w") as f:
        f.write(SHIM)
    subprocess.run([os.environ.get("NVCC", "nvcc"), "-gencode", "arch=compute_103a,code=sm_103a", "-O3", "-std=c++17",
                    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden", "-shared", "--threads", "0",
                    f"-DMOE_TC_WAIT_CYCLES={request.param}", "-I", CSRC, shim, os.path.join(CSRC, "fp4_linear.cu"),
                    os.path.join(CSRC, "route.cu"), os.path.join(CSRC, "tc_host.cu"), "-o", lib], check=True)
    lib = C.CDLL(lib)
    lib.cycles = request.param
    lib.product.argtypes = [C.c_int] + [C.c_void_p] * 4 + [C.c_int] * 3 + [C.c_void_p] * 3
    lib.logits.argtypes = [C.c_void_p] * 2 + [C.c_int] * 3 + [C.c_void_p] * 3
    return lib


# one CTA a tile, pairs, tokens as columns, scales by shifted loads; a few tiles or many each
WHOLE = [(1, 131072, 256), (128, 40000, 256), (600, 20000, 64), (2048, 8192, 4096), (8192, 2048, 512),
         (300, 40000, 544), (4000, 4000, 2080)]
# K in two or four parts, on a cluster: rows as rows or as columns, pairs, shifted scales
SPLIT = [(1, 4096, 4096), (16, 2048, 2048), (64, 1536, 2048), (100, 640, 4096), (128, 128, 8192), (200, 2048, 544),
         (600, 1536, 2048), (512, 3000, 4096)]


@pytest.mark.parametrize("nv", [True, False])
@pytest.mark.parametrize("B,N,K", WHOLE + SPLIT)
def test_a_wait_that_runs_out(m, impatient, nv, B, N, K):  # noqa: F811
    r = np.random.default_rng([B, N, K])
    lo, hi, blk = (0x20, 0x40, 16) if nv else (118, 130, 32)
    a = [dev(r.integers(0, 256, (n, K // 2)).astype(np.uint8)) for n in (B, N)]
    s = [dev(r.integers(lo, hi, (n, K // blk)).astype(np.uint8)) for n in (B, N)]
    st = torch.zeros(1, dtype=torch.int64, device="cuda")
    fmt = m.MOE_W_NVFP4 if nv else m.MOE_W_MXFP4

    def full():
        out = torch.full((B, N), float("nan"), device="cuda")
        st.zero_()
        m.moe_fp4_linear(fmt, a[0], s[0], None, a[1], s[1], None, B, N, K, out, m.MOE_T_F32, d_status=st)
        assert st.item() == 0
        return out

    want = full()
    gave_up = 0
    for _ in range(4):
        out = torch.full((B, N), float("nan"), device="cuda")
        st.zero_()
        rc = impatient.product(int(nv), a[0].data_ptr(), s[0].data_ptr(), a[1].data_ptr(), s[1].data_ptr(), B, N, K,
                               out.data_ptr(), st.data_ptr(), torch.cuda.current_stream().cuda_stream)
        assert rc == 0
        torch.cuda.synchronize()  # the context is as it was
        untouched = out.isnan()
        assert torch.equal(out[~untouched], want[~untouched])
        assert st.item() == m.MOE_STATUS_TIMEOUT if untouched.any() else st.item() in (0, m.MOE_STATUS_TIMEOUT)
        gave_up += int(st.item() != 0)
    if impatient.cycles == 0:
        assert gave_up  # the first copy takes longer
    print(f"{B} x {N} x {K}: {gave_up} of 4 gave up, {untouched.double().mean().item():.3f} untouched in the last")
    assert torch.equal(full(), want)  # tensor memory and barriers were left as they should be
    x = ref.decode(a[0][-1:].cpu().numpy(), s[0][-1:].cpu().numpy(), nv)
    w = ref.decode(a[1][:64].cpu().numpy(), s[1][:64].cpu().numpy(), nv)
    err = np.abs(want[-1:, :64].double().cpu().numpy() - x @ w.T)
    assert (err <= (K / 32 + 40) * 2 * U * (np.abs(x) @ np.abs(w).T)).all()


# the router's bf16 tiles: one CTA, split in two and four, pairs, pairs split
@pytest.mark.parametrize("B,H,E", [(20500, 256, 64), (40000, 128, 100), (16, 2048, 512), (64, 4096, 384), (600, 2048, 1024),
                                   (8192, 4096, 256), (20000, 512, 700)])
def test_a_wait_of_the_router_that_runs_out(m, impatient, B, H, E):  # noqa: F811
    r = np.random.default_rng([B, H, E])
    x = dev(r.normal(0, 1, (B, H)).astype(np.float32)).bfloat16()
    router = dev(r.normal(0, H ** -0.5, (E, H)).astype(np.float32)).bfloat16()
    ids, w = torch.empty(B, 1, dtype=torch.int32, device="cuda"), torch.empty(B, 1, device="cuda")
    st = torch.zeros(1, dtype=torch.int64, device="cuda")

    def full():
        z = torch.full((B, E), float("nan"), device="cuda")
        st.zero_()
        m.moe_route(x, router, None, B, H, E, 1, z, ids, w, d_status=st)
        assert st.item() == 0
        return z

    want = full()
    gave_up = 0
    for _ in range(4):
        z = torch.full((B, E), float("nan"), device="cuda")
        st.zero_()
        assert impatient.logits(x.data_ptr(), router.data_ptr(), B, H, E, z.data_ptr(), st.data_ptr(),
                                torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        untouched = z.isnan()
        assert torch.equal(z[~untouched], want[~untouched])
        assert st.item() == m.MOE_STATUS_TIMEOUT if untouched.any() else st.item() in (0, m.MOE_STATUS_TIMEOUT)
        gave_up += int(st.item() != 0)
    if impatient.cycles == 0:
        assert gave_up
    print(f"router {B} x {H} x {E}: {gave_up} of 4 gave up, {untouched.double().mean().item():.3f} untouched in the last")
    assert torch.equal(full(), want)
    size = x.double().abs() @ router.double().abs().T
    assert ((want.double() - x.double() @ router.double().T).abs() <= (H / 16 + 40) * 2 * U * size).all()

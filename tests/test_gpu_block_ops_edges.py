"""The operators around the experts where buffers are used again, calls follow each
other without a stop, and values or sizes are extreme.  Tolerances as in
test_gpu_block_ops.py."""
import numpy as np
import pytest
import torch

from tests import block_ref as ref
from tests.test_gpu_block_ops import U, dev, fmt_of, m  # noqa: F401  (m: the library)

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

// fp4_linear.cu -- the product of two 4-bit matrices (formulas in moe_cache.h):
// block-scaled tcgen05 MMAs over packed e2m1, tile_gemm.cuh.
//
// P are the tokens and Q the weights, or, with up to 64 tokens, the other way round
// (NT = 16, 32 or 64: a tile's MMAs cost no more than its Q rows): the tile is the one
// estimated to take least.  The weights as P where their 128-row tiles fill the SMs
// (64 x 70,000 x 2,048: 17.2 us, as Q 21.8) or K is long enough to split (32 x 4,096 x
// 4,096: 6.6 and 8.0), as Q between (64 x 8,192 x 2,048: 5.9 us, as P 8.3).
#include "block_ops.cuh"
#include "tile_gemm.cuh"

namespace moe {
namespace {

template <tg::Kind KIND>
cudaError_t by_rows(const Fp4Linear& l, int sms, cudaStream_t s) {
  const long long c64 = tg::cycles<KIND, 64, 1>(l.rows, l.n, l.k, sms),
                  c128 = tg::cycles<KIND, 128, 1>(l.rows, l.n, l.k, sms),
                  c192 = tg::cycles<KIND, 192, 2>(l.rows, l.n, l.k, sms);
  long long best = c64 < c128 ? c64 : c128;
  best = c192 < best ? c192 : best;
  const long long turned = l.rows <= 16   ? tg::cycles<KIND, 16, 1>(l.n, l.rows, l.k, sms)
                           : l.rows <= 32 ? tg::cycles<KIND, 32, 1>(l.n, l.rows, l.k, sms)
                                          : tg::cycles<KIND, 64, 1>(l.n, l.rows, l.k, sms);
  const bool swap = l.rows <= 64 && turned <= best;
  tg::Problem p{};
  p.p = swap ? l.wc : l.xc;
  p.q = swap ? l.xc : l.wc;
  p.ps = swap ? l.ws : l.xs;
  p.qs = swap ? l.xs : l.ws;
  p.p_rows = swap ? l.n : l.rows;
  p.q_rows = swap ? l.rows : l.n;
  p.p_stride = p.q_stride = l.k / 2;
  p.k = l.k;
  p.g0 = l.xg;
  p.g1 = l.wg;
  p.out = l.out;
  p.out_stride = l.out_stride;
  p.f32 = l.f32;
  p.status = l.status;
  if (swap) {
    if (l.rows <= 16) return tg::launch<KIND, 16, 1, true>(p, sms, s);
    if (l.rows <= 32) return tg::launch<KIND, 32, 1, true>(p, sms, s);
    return tg::launch<KIND, 64, 1, true>(p, sms, s);
  }
  if (c192 == best) return tg::launch<KIND, 192, 2, false>(p, sms, s);
  if (c128 == best) return tg::launch<KIND, 128, 1, false>(p, sms, s);
  return tg::launch<KIND, 64, 1, false>(p, sms, s);
}

}  // namespace

cudaError_t launch_fp4_linear(const Fp4Linear& l, cudaStream_t s) {
  tc::DeviceInfo d;
  const cudaError_t e = tc::device_info(&d);
  if (e != cudaSuccess) return e;
  return l.nv ? by_rows<tg::kNv>(l, d.sms, s) : by_rows<tg::kMx>(l, d.sms, s);
}

}  // namespace moe

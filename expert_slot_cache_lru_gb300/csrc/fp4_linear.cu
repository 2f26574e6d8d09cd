// fp4_linear.cu -- the product of two 4-bit matrices (formulas in moe_cache.h).
#include "block_ops.cuh"
#include "fp4.cuh"
#include "tile_dot.cuh"

namespace moe {
namespace {

template <bool NV>
struct Fp4Rows {
  const uint8_t *codes, *scales;
  int k;
  __device__ float operator()(int r, int i) const {
    constexpr int BLK = NV ? 16 : 32;
    const size_t at = (size_t)r * k + i;
    const float2 q = e2m1x2_to_f(codes[at / 2]);
    const uint32_t s = scales[at / BLK];
    return ((i & 1) ? q.y : q.x) * (NV ? e4m3_to_f(s) : e8m0_to_f(s));
  }
};
template <typename T>
struct StoreScaled {
  T* p;
  long long stride;
  const float *xg, *wg;
  __device__ void operator()(int m, int n, float v) const {
    v *= (xg ? *xg : 1.f) * (wg ? *wg : 1.f);
    if constexpr (sizeof(T) == 4) p[m * stride + n] = v;
    else p[m * stride + n] = __float2bfloat16_rn(v);
  }
};

template <bool NV, typename T>
cudaError_t simple(const Fp4Linear& a, cudaStream_t s) {
  for (long long r0 = 0; r0 < a.rows; r0 += 65535 * 64) {
    const int n = (int)(a.rows - r0 < 65535 * 64 ? a.rows - r0 : 65535 * 64);
    constexpr int BLK = NV ? 16 : 32;
    tile_dot_kernel<<<dim3((a.n + 63) / 64, (n + 63) / 64), 256, 0, s>>>(
        Fp4Rows<NV>{a.xc + r0 * (a.k / 2), a.xs + r0 * (a.k / BLK), a.k},
        Fp4Rows<NV>{a.wc, a.ws, a.k},
        StoreScaled<T>{static_cast<T*>(a.out) + r0 * a.out_stride, a.out_stride, a.xg, a.wg}, n,
        a.n, a.k);
  }
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_fp4_linear(const Fp4Linear& a, cudaStream_t s) {
  if (a.nv) return a.f32 ? simple<true, float>(a, s) : simple<true, __nv_bfloat16>(a, s);
  return a.f32 ? simple<false, float>(a, s) : simple<false, __nv_bfloat16>(a, s);
}

}  // namespace moe

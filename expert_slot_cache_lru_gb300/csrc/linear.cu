// linear.cu -- the bf16 products (formulas in moe_cache.h): which kernel takes a
// call, and the CUDA-core tiles for operands of any layout.
//
// Tiles of 64 rows x 64 results (of both matrices if gated), 4 x 4 results per thread, operands through
// shared memory as fp32: bound by its FMAs.
#include "linear.cuh"
#include "tc.cuh"

namespace moe {
namespace {

using namespace lin;

template <bool GATED>
__global__ void __launch_bounds__(256) tile_kernel(const Linear l, int tn) {
  constexpr int M = GATED ? 2 : 1;
  __shared__ float xs[32][65], ws[M][32][65];
  __shared__ int src[64];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  tc::pdl_trigger();
  tc::pdl_wait();
  Walk walk;
  walk.start(l, 6, 1, tn);
  Tile t;
  for (long long i = blockIdx.x; i < 0x40000000 && walk.seek((int)i, t); i += gridDim.x) {
    const long long n0 = t.n * 64ll;
    const __nv_bfloat16* w = l.w + t.group * l.group_stride;
    __syncthreads();
    if (threadIdx.x < 64) src[threadIdx.x] = (int)threadIdx.x < t.rows ? source_row(l, t.row + threadIdx.x) : -1;
    __syncthreads();
    float acc[M][4][4] = {};
    for (long long k0 = 0; k0 < l.k; k0 += 32) {
      for (int j = threadIdx.x; j < 64 * 32; j += 256) {
        const int r = j >> 5, k = j & 31;
        const bool in = k0 + k < l.k;
        xs[k][r] = in && src[r] >= 0 ? __bfloat162float(l.x[src[r] * l.x_stride + k0 + k]) : 0.f;
#pragma unroll
        for (int m = 0; m < M; ++m)
          ws[m][k][r] = in && n0 + r < l.n
                            ? __bfloat162float(w[(m * (long long)l.n + n0 + r) * l.w_stride + k0 + k])
                            : 0.f;
      }
      __syncthreads();
#pragma unroll 8
      for (int k = 0; k < 32; ++k) {
        float xv[4];
#pragma unroll
        for (int a = 0; a < 4; ++a) xv[a] = xs[k][ty + 16 * a];
#pragma unroll
        for (int m = 0; m < M; ++m)
#pragma unroll
          for (int b = 0; b < 4; ++b) {
            const float wv = ws[m][k][tx + 16 * b];
#pragma unroll
            for (int a = 0; a < 4; ++a) acc[m][a][b] = fmaf(xv[a], wv, acc[m][a][b]);
          }
      }
      __syncthreads();
    }
    with_act(l.act, [&](auto act) {
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const long long n = n0 + tx + 16 * b;
        if (n >= l.n) continue;
        float bias[M] = {};
        if (l.bias)
#pragma unroll
          for (int m = 0; m < M; ++m)
            bias[m] = __bfloat162float(l.bias[((long long)t.group * M + m) * l.n + n]);
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          const int r = ty + 16 * a;
          if (src[r] < 0) continue;
          float y = act(acc[0][a][b] + bias[0]);
          if (GATED) y *= acc[M - 1][a][b] + bias[M - 1];
          finish(l, t.row + r, n, y);
        }
      }
    });
  }
}

template <bool GATED>
cudaError_t launch_tiles(const Linear& l, int sms, cudaStream_t s) {
  const int tn = (int)((l.n + 63ll) / 64);
  const long long most = most_tiles(l, 6, tn);
  if (most > 0x3fffffff) return cudaErrorInvalidValue;
  const long long grid = most < 8ll * sms ? most : 8ll * sms;
  return tc::launch_early(tile_kernel<GATED>, dim3((unsigned)grid), dim3(256), 0, s, l, tn);
}

}  // namespace

cudaError_t launch_linear(const Linear& l, cudaStream_t s) {
  tc::DeviceInfo d;
  const cudaError_t e = tc::device_info(&d);
  if (e != cudaSuccess) return e;
  const bool whole = l.k % 8 == 0 && l.x_stride % 8 == 0 && l.w_stride % 8 == 0 && l.group_stride % 8 == 0 &&
                     ((reinterpret_cast<uintptr_t>(l.x) | reinterpret_cast<uintptr_t>(l.w)) & 15) == 0;
  // gathered rows are addressed in 32 bits of 16-byte pieces
  const bool near = !l.order || (double)l.x_rows * l.x_stride / 8 < 4294967296.0;
  if (whole && near && (!l.gated || l.n % 16 == 0)) return launch_linear_tc(l, d.sms, s);
  return l.gated ? launch_tiles<true>(l, d.sms, s) : launch_tiles<false>(l, d.sms, s);
}

}  // namespace moe

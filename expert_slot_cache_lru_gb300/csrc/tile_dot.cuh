// tile_dot.cuh -- c[m][n] = sum_k a[m][k] b[n][k] in fp32 on the CUDA cores, for
// any sizes and element types: 64 x 64 tiles, 4 x 4 results per thread.  A and B
// return element (row, k) as a float, C stores one result.
#pragma once

#include <cuda_runtime.h>

namespace moe {

template <typename A, typename B, typename C>
__global__ void __launch_bounds__(256) tile_dot_kernel(A a, B b, C c, int M, int N, int K) {
  __shared__ float as[32][65], bs[32][65];
  const long long m0 = (long long)blockIdx.y * 64;
  const int n0 = blockIdx.x * 64, tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  float acc[4][4] = {};
  for (int k0 = 0; k0 < K; k0 += 32) {
    for (int i = threadIdx.x; i < 64 * 32; i += 256) {
      const int r = i >> 5, k = i & 31;
      as[k][r] = m0 + r < M && k0 + k < K ? a((int)m0 + r, k0 + k) : 0.f;
      bs[k][r] = n0 + r < N && k0 + k < K ? b(n0 + r, k0 + k) : 0.f;
    }
    __syncthreads();
#pragma unroll 8
    for (int k = 0; k < 32; ++k) {
      float av[4], bv[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        av[i] = as[k][ty + 16 * i];
        bv[i] = bs[k][tx + 16 * i];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(av[i], bv[j], acc[i][j]);
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const long long m = m0 + ty + 16 * i;
      const int n = n0 + tx + 16 * j;
      if (m < M && n < N) c((int)m, n, acc[i][j]);
    }
}

}  // namespace moe

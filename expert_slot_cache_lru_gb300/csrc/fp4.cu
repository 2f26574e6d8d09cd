// fp4.cu -- conversions between matrices and the 4-bit banks of an expert blob
// (formulas and layouts in moe_cache.h).
#include "block_ops.cuh"
#include "fp4.cuh"

namespace moe {
namespace {

__device__ __forceinline__ float load_f(const float* p) { return *p; }
__device__ __forceinline__ float load_f(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store_f(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_f(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

constexpr int kThreads = 256;

// one thread per block
template <bool NV, typename T>
__global__ void __launch_bounds__(kThreads)
quantize_kernel(const T* src, long long stride, int rows, int nb, const float* g, uint8_t* codes,
                uint8_t* scales) {
  constexpr int BLK = NV ? 16 : 32;
  const float gl = g ? *g : 1.f;
  const long long n = (long long)rows * nb;
  for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < n;
       i += (long long)gridDim.x * kThreads) {
    const long long r = i / nb;
    const T* p = src + r * stride + (i - r * nb) * BLK;
    float v[BLK], amax = 0.f;
    bool nan = false;
#pragma unroll
    for (int j = 0; j < BLK; ++j) {
      v[j] = load_f(p + j);
      amax = fmaxf(amax, fabsf(v[j]));
      nan |= v[j] != v[j];
    }
    uint32_t sb;
    float step;
    if (NV) {
      sb = f_to_e4m3(fminf(amax / (6.f * gl), 448.f));
      step = e4m3_to_f(sb) * gl;
    } else {
      // floor(log2 amax) of a normal number is its exponent field - 127; the
      // scales below 2^-127 that a smaller amax asks for are clamped anyway
      const int ex = (int)(__float_as_uint(amax) >> 23) - 2;
      sb = (uint32_t)min(max(ex, 0), 254);
      step = e8m0_to_f(sb);
    }
    if (nan) sb = NV ? 0x7fu : 0xffu;
    scales[i] = (uint8_t)sb;
    const bool zero = nan || !(step > 0.f);
#pragma unroll
    for (int j = 0; j < BLK; j += 2)
      codes[i * (BLK / 2) + j / 2] =
          zero ? 0u : (uint8_t)f_to_e2m1x2(v[j] / step, v[j + 1] / step);
  }
}

template <bool NV, typename T>
__global__ void __launch_bounds__(kThreads)
dequantize_kernel(const uint8_t* codes, const uint8_t* scales, int rows, int nb, const float* g,
                  T* dst, long long stride) {
  constexpr int BLK = NV ? 16 : 32;
  const float gl = g ? *g : 1.f;
  const long long n = (long long)rows * nb;
  for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < n;
       i += (long long)gridDim.x * kThreads) {
    const long long r = i / nb;
    T* p = dst + r * stride + (i - r * nb) * BLK;
    const float s = NV ? e4m3_to_f(scales[i]) : e8m0_to_f(scales[i]);
#pragma unroll
    for (int j = 0; j < BLK; j += 2) {
      const float2 q = e2m1x2_to_f(codes[i * (BLK / 2) + j / 2]);
      store_f(p + j, q.x * s * gl);
      store_f(p + j + 1, q.y * s * gl);
    }
  }
}

// the bits of the largest finite magnitude (nonnegative floats order as integers)
template <typename T>
__global__ void __launch_bounds__(kThreads)
amax_kernel(const T* src, long long stride, int rows, int cols, unsigned* out) {
  const long long n = (long long)rows * cols;
  unsigned m = 0;
  for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < n;
       i += (long long)gridDim.x * kThreads) {
    const long long r = i / cols;
    const unsigned u = __float_as_uint(load_f(src + r * stride + (i - r * cols))) & 0x7fffffffu;
    if (u < 0x7f800000u) m = max(m, u);
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0 && m) atomicMax(out, m);
}
__global__ void global_kernel(float* g) {
  const float m = *g;
  *g = m > 0.f ? fmaxf(m / 2688.f, 1.17549435e-38f) : 1.f;
}

int grid_for(long long n) {
  const long long c = (n + kThreads - 1) / kThreads;
  return (int)(c < 152 * 16 ? c : 152 * 16);
}

}  // namespace

cudaError_t launch_fp4_quantize(bool nv, const void* src, int dtype, long long stride, int rows,
                                int cols, const float* g, uint8_t* codes, uint8_t* scales,
                                cudaStream_t s) {
  const int nb = cols / (nv ? 16 : 32), grid = grid_for((long long)rows * nb);
  auto go = [&](auto kern, auto* p) {
    kern<<<grid, kThreads, 0, s>>>(p, stride, rows, nb, g, codes, scales);
    return cudaGetLastError();
  };
  if (dtype == MOE_T_F32) {
    auto* p = static_cast<const float*>(src);
    return nv ? go(quantize_kernel<true, float>, p) : go(quantize_kernel<false, float>, p);
  }
  auto* p = static_cast<const __nv_bfloat16*>(src);
  return nv ? go(quantize_kernel<true, __nv_bfloat16>, p) : go(quantize_kernel<false, __nv_bfloat16>, p);
}

cudaError_t launch_fp4_dequantize(bool nv, const uint8_t* codes, const uint8_t* scales,
                                  const float* g, int rows, int cols, void* dst, int dtype,
                                  long long stride, cudaStream_t s) {
  const int nb = cols / (nv ? 16 : 32), grid = grid_for((long long)rows * nb);
  auto go = [&](auto kern, auto* p) {
    kern<<<grid, kThreads, 0, s>>>(codes, scales, rows, nb, g, p, stride);
    return cudaGetLastError();
  };
  if (dtype == MOE_T_F32) {
    auto* p = static_cast<float*>(dst);
    return nv ? go(dequantize_kernel<true, float>, p) : go(dequantize_kernel<false, float>, p);
  }
  auto* p = static_cast<__nv_bfloat16*>(dst);
  return nv ? go(dequantize_kernel<true, __nv_bfloat16>, p)
            : go(dequantize_kernel<false, __nv_bfloat16>, p);
}

cudaError_t launch_fp4_global_scale(const void* src, int dtype, long long stride, int rows,
                                    int cols, float* g, cudaStream_t s) {
  const cudaError_t e = cudaMemsetAsync(g, 0, sizeof(float), s);
  if (e != cudaSuccess) return e;
  const int grid = grid_for((long long)rows * cols);
  unsigned* u = reinterpret_cast<unsigned*>(g);
  if (dtype == MOE_T_F32)
    amax_kernel<<<grid, kThreads, 0, s>>>(static_cast<const float*>(src), stride, rows, cols, u);
  else
    amax_kernel<<<grid, kThreads, 0, s>>>(static_cast<const __nv_bfloat16*>(src), stride, rows, cols, u);
  global_kernel<<<1, 1, 0, s>>>(g);
  return cudaGetLastError();
}

}  // namespace moe

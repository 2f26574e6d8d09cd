// fp4.cu -- conversions between matrices and the 4-bit banks of an expert blob
// (formulas and layouts in moe_cache.h).
//
// Bound by memory: 2 or 4 bytes in, 0.53 to 0.56 out per element (and back).
// One thread owns 16 neighbouring elements: an NVFP4 block, or half an MXFP4 block
// whose maximum it shares with its neighbour; a warp reads 1 or 2 KB and writes
// 256 bytes of codes without gaps, with 32-byte loads and stores where the rows
// allow them.  kUnits such pieces per thread are loaded before the first is used
// where there is work for every SM; small matrices take one.
// Quotients x / (s g): correctly rounded in three operations from one reciprocal
// per block, q = x r, q' = q + r (x - q d) with r the correctly rounded 1 / d
// (Markstein, IBM J. Res. Dev. 34, 1990); a block whose divisor or maximum is
// near the ends of fp32's range divides instead.
#include <type_traits>

#include "block_ops.cuh"
#include "fp4.cuh"
#include "tc.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 4;

// ---------------------------------------------------------------- loads and stores
__device__ __forceinline__ void ld32(const void* p, uint32_t (&w)[8]) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
      : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
      : "l"(p));
}
__device__ __forceinline__ void st32(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
__device__ __forceinline__ float lo_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// 16 elements as loaded (bf16: 8 words, fp32: 16)
template <typename T>
struct Raw {
  uint32_t w[sizeof(T) == 4 ? 16 : 8];
};
template <bool VEC>
__device__ __forceinline__ void load16(const float* p, Raw<float>& r) {
  if (VEC) {
    uint32_t a[8], b[8];
    ld32(p, a);
    ld32(p + 8, b);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      r.w[i] = a[i];
      r.w[8 + i] = b[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) r.w[i] = __float_as_uint(p[i]);
  }
}
template <bool VEC>
__device__ __forceinline__ void load16(const __nv_bfloat16* p, Raw<__nv_bfloat16>& r) {
  if (VEC) {
    ld32(p, r.w);
  } else {
    const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
    for (int i = 0; i < 8; ++i) r.w[i] = h[2 * i] | (uint32_t)h[2 * i + 1] << 16;
  }
}
__device__ __forceinline__ float elem(const Raw<float>& r, int i) { return __uint_as_float(r.w[i]); }
__device__ __forceinline__ float elem(const Raw<__nv_bfloat16>& r, int i) {
  return i & 1 ? hi_bf16(r.w[i / 2]) : lo_bf16(r.w[i / 2]);
}
template <bool VEC>
__device__ __forceinline__ void store16(float* p, const float (&v)[16]) {
  if (VEC) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[8 * h + i]);
      st32(p + 8 * h, w);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) p[i] = v[i];
  }
}
template <bool VEC>
__device__ __forceinline__ void store16(__nv_bfloat16* p, const float (&v)[16]) {
  if (VEC) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    st32(p, w);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) p[i] = __float2bfloat16_rn(v[i]);
  }
}

// maximum that lets a NaN through
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// ---------------------------------------------------------------- quantize
// one piece: the codes of 16 elements, the block's scale byte
template <bool NV, typename T>
__device__ __forceinline__ uint2 quantize16(const Raw<T>& x, float g, uint32_t& sb) {
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) amax = max_nan(amax, fabsf(elem(x, i)));
  float step;
  if (NV) {
    sb = f_to_e4m3(fminf(amax / (6.f * g), 448.f));
    step = e4m3_to_f(sb) * g;
  } else {
    amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    // floor(log2 amax) of a normal number is its exponent field - 127; the
    // scales below 2^-127 that a smaller amax asks for are clamped anyway
    const int ex = (int)(__float_as_uint(amax) >> 23) - 2;
    sb = (uint32_t)min(max(ex, 0), 254);
    step = e8m0_to_f(sb);
  }
  uint32_t c[8];
  if (amax != amax) {
    sb = NV ? 0x7fu : 0xffu;
    return make_uint2(0u, 0u);
  }
  if (!(step > 0.f)) return make_uint2(0u, 0u);
  if (!NV && sb > 0 && sb < 253) {
    const float r = __uint_as_float((254u - sb) << 23);  // 1 / step, exact: so are the quotients
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = f_to_e2m1x2(elem(x, 2 * i) * r, elem(x, 2 * i + 1) * r);
  } else if (NV && step > 1e-18f && step < 1e18f && amax < 1e19f) {
    const float r = 1.f / step;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float q[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float v = elem(x, 2 * i + j), q0 = v * r;
        q[j] = copysignf(fmaf(fmaf(-q0, step, v), r, q0), v);  // the sums lose a zero's sign
      }
      c[i] = f_to_e2m1x2(q[0], q[1]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = f_to_e2m1x2(elem(x, 2 * i) / step, elem(x, 2 * i + 1) / step);
  }
  return make_uint2(c[0] | c[1] << 8 | c[2] << 16 | c[3] << 24,
                    c[4] | c[5] << 8 | c[6] << 16 | c[7] << 24);
}

// np pieces of 16 per row; rows without gaps arrive as one long row.  Rows count without
// sign: up to 2^31 - 1 plus the grid's at most 65,535 stays below 2^32 (64-bit rows: 213
// us where these take 210, 131,072 x 2,048 and back).
template <bool NV, typename T, bool VEC, int U>
__global__ void __launch_bounds__(kThreads)
quantize_kernel(const T* src, long long stride, int rows, long long np, const float* gp,
                uint8_t* codes, uint8_t* scales) {
  tc::pdl_trigger();
  tc::pdl_wait();
  const float g = NV && gp ? *gp : 1.f;
  const long long i0 = (long long)blockIdx.x * (kThreads * U) + threadIdx.x;
  for (unsigned row = blockIdx.y; row < (unsigned)rows; row += gridDim.y) {
    const T* p = src + row * stride;
    Raw<T> x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long i = i0 + u * kThreads;
      if (i < np) load16<VEC>(p + i * 16, x[u]);
      else x[u] = Raw<T>{};
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long i = i0 + u * kThreads, at = row * np + i;
      uint32_t sb;
      const uint2 c = quantize16<NV, T>(x[u], g, sb);  // every lane: MXFP4 exchanges maxima
      if (i < np) {
        *reinterpret_cast<uint2*>(codes + at * 8) = c;
        if (NV) scales[at] = (uint8_t)sb;
        else if (!(i & 1)) scales[at / 2] = (uint8_t)sb;
      }
    }
  }
}

// ---------------------------------------------------------------- dequantize
template <bool NV, typename T, bool VEC, int U>
__global__ void __launch_bounds__(kThreads)
dequantize_kernel(const uint8_t* codes, const uint8_t* scales, int rows, long long np,
                  const float* gp, T* dst, long long stride) {
  tc::pdl_trigger();
  tc::pdl_wait();
  const float g = NV && gp ? *gp : 1.f;
  const long long i0 = (long long)blockIdx.x * (kThreads * U) + threadIdx.x;
  for (unsigned row = blockIdx.y; row < (unsigned)rows; row += gridDim.y) {
    T* p = dst + row * stride;
    uint2 c[U];
    uint32_t sb[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long i = i0 + u * kThreads, at = row * np + i;
      if (i < np) {
        c[u] = *reinterpret_cast<const uint2*>(codes + at * 8);
        sb[u] = scales[NV ? at : at / 2];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long i = i0 + u * kThreads;
      if (i >= np) continue;
      const float s = NV ? e4m3_to_f(sb[u]) : e8m0_to_f(sb[u]);
      float v[16];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 q = e2m1x2_to_f(((j < 4 ? c[u].x : c[u].y) >> (8 * (j & 3))) & 0xffu);
        v[2 * j] = q.x * s * g;
        v[2 * j + 1] = q.y * s * g;
      }
      store16<VEC>(p + i * 16, v);
    }
  }
}

// ---------------------------------------------------------------- global scale
// the bits of the largest finite magnitude (nonnegative floats order as integers);
// VEC: pieces of 16 elements, else single ones
__device__ __forceinline__ unsigned finite_bits(float v) {
  const unsigned u = __float_as_uint(v) & 0x7fffffffu;
  return u < 0x7f800000u ? u : 0u;
}
template <typename T, bool VEC>
__global__ void __launch_bounds__(kThreads)
amax_kernel(const T* src, long long stride, int rows, long long cols, unsigned* out) {
  unsigned m = 0;
  for (unsigned row = blockIdx.y; row < (unsigned)rows; row += gridDim.y)
    for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < cols;
         i += (long long)gridDim.x * kThreads) {
      if constexpr (VEC) {
        Raw<T> x;
        load16<true>(src + row * stride + i * 16, x);
#pragma unroll
        for (int j = 0; j < 16; ++j) m = max(m, finite_bits(elem(x, j)));
      } else {
        m = max(m, finite_bits((float)src[row * stride + i]));
      }
    }
  m = __reduce_max_sync(0xffffffffu, m);
  if ((threadIdx.x & 31) == 0 && m) atomicMax(out, m);
}
__global__ void global_kernel(float* g) {
  const float m = *g;
  *g = m > 0.f ? fmaxf(m / 2688.f, 1.17549435e-38f) : 1.f;
}

// ---------------------------------------------------------------- launches
bool aligned32(const void* p, long long stride_bytes) {
  return ((reinterpret_cast<uintptr_t>(p) | (uintptr_t)stride_bytes) & 31) == 0;
}
// Rows without gaps are one row.  kUnits pieces per thread once that still
// fills the SMs twice over.
struct Grid {
  dim3 grid;
  int rows;
  long long width;
  bool wide;
};
Grid grid_for(int rows, long long width, bool whole, int per_thread, int sms) {
  Grid g;
  g.rows = whole ? 1 : rows;
  g.width = whole ? rows * width : width;
  g.wide = (long long)rows * width >= 2LL * sms * kThreads * per_thread &&
           g.width >= (long long)kThreads * per_thread;
  const long long per = (long long)kThreads * (g.wide ? per_thread : 1);
  g.grid = dim3((unsigned)((g.width + per - 1) / per), (unsigned)(g.rows < 65535 ? g.rows : 65535));
  return g;
}

template <bool NV, typename T>
cudaError_t quantize(const T* src, long long stride, int rows, int cols, const float* g,
                     uint8_t* codes, uint8_t* scales, cudaStream_t s) {
  tc::DeviceInfo d;
  const cudaError_t e = tc::device_info(&d);
  if (e != cudaSuccess) return e;
  const bool vec = aligned32(src, stride * (long long)sizeof(T));
  const Grid q = grid_for(rows, cols / 16, stride == cols, vec ? kUnits : 1, d.sms);
  auto go = [&](auto kern) {
    return tc::launch_early(kern, q.grid, dim3(kThreads), 0, s, src, stride, q.rows, q.width, g, codes, scales);
  };
  if (!vec) return go(quantize_kernel<NV, T, false, 1>);
  return q.wide ? go(quantize_kernel<NV, T, true, kUnits>) : go(quantize_kernel<NV, T, true, 1>);
}
template <bool NV, typename T>
cudaError_t dequantize(const uint8_t* codes, const uint8_t* scales, const float* g, int rows,
                       int cols, T* dst, long long stride, cudaStream_t s) {
  tc::DeviceInfo d;
  const cudaError_t e = tc::device_info(&d);
  if (e != cudaSuccess) return e;
  const bool vec = aligned32(dst, stride * (long long)sizeof(T));
  const Grid q = grid_for(rows, cols / 16, stride == cols, vec ? kUnits : 1, d.sms);
  auto go = [&](auto kern) {
    return tc::launch_early(kern, q.grid, dim3(kThreads), 0, s, codes, scales, q.rows, q.width, g, dst, stride);
  };
  if (!vec) return go(dequantize_kernel<NV, T, false, 1>);
  return q.wide ? go(dequantize_kernel<NV, T, true, kUnits>) : go(dequantize_kernel<NV, T, true, 1>);
}

}  // namespace

cudaError_t launch_fp4_quantize(bool nv, const void* src, int dtype, long long stride, int rows,
                                int cols, const float* g, uint8_t* codes, uint8_t* scales,
                                cudaStream_t s) {
  if (dtype == MOE_T_F32) {
    auto* p = static_cast<const float*>(src);
    return nv ? quantize<true>(p, stride, rows, cols, g, codes, scales, s)
              : quantize<false>(p, stride, rows, cols, g, codes, scales, s);
  }
  auto* p = static_cast<const __nv_bfloat16*>(src);
  return nv ? quantize<true>(p, stride, rows, cols, g, codes, scales, s)
            : quantize<false>(p, stride, rows, cols, g, codes, scales, s);
}

cudaError_t launch_fp4_dequantize(bool nv, const uint8_t* codes, const uint8_t* scales,
                                  const float* g, int rows, int cols, void* dst, int dtype,
                                  long long stride, cudaStream_t s) {
  if (dtype == MOE_T_F32) {
    auto* p = static_cast<float*>(dst);
    return nv ? dequantize<true>(codes, scales, g, rows, cols, p, stride, s)
              : dequantize<false>(codes, scales, g, rows, cols, p, stride, s);
  }
  auto* p = static_cast<__nv_bfloat16*>(dst);
  return nv ? dequantize<true>(codes, scales, g, rows, cols, p, stride, s)
            : dequantize<false>(codes, scales, g, rows, cols, p, stride, s);
}

cudaError_t launch_fp4_global_scale(const void* src, int dtype, long long stride, int rows,
                                    int cols, float* g, cudaStream_t s) {
  tc::DeviceInfo d;
  cudaError_t e = tc::device_info(&d);
  if (e == cudaSuccess) e = cudaMemsetAsync(g, 0, sizeof(float), s);
  if (e != cudaSuccess) return e;
  unsigned* u = reinterpret_cast<unsigned*>(g);
  auto go = [&](auto* p) {
    using T = std::remove_const_t<std::remove_pointer_t<decltype(p)>>;
    const bool vec = cols % 16 == 0 && aligned32(src, stride * (long long)sizeof(T));
    Grid q = grid_for(rows, vec ? cols / 16 : cols, stride == cols, 1, d.sms);
    const unsigned most = q.rows > 8 ? d.sms : d.sms * 8;  // CTAs loop over what is left
    if (q.grid.x > most) q.grid.x = most;
    if (q.grid.y > 1024) q.grid.y = 1024;
    if (vec) amax_kernel<T, true><<<q.grid, kThreads, 0, s>>>(p, stride, q.rows, q.width, u);
    else amax_kernel<T, false><<<q.grid, kThreads, 0, s>>>(p, stride, q.rows, q.width, u);
  };
  if (dtype == MOE_T_F32) go(static_cast<const float*>(src));
  else go(static_cast<const __nv_bfloat16*>(src));
  global_kernel<<<1, 1, 0, s>>>(g);
  return cudaGetLastError();
}

}  // namespace moe

// block_norm.cu -- the seam between two blocks: post-norm, gate, residual add
// and the next block's pre-norm in one pass (formulas in moe_cache.h).
//
// Bound by memory: h and y are read once and h' and x' written once; a row stays
// in its CTA's registers (fp32) between the two sums, so h_out may be h itself.
//
// ring_kernel, a bf16 residual with more rows of whole 16-byte pieces (up to 8,192
// elements) than the SMs hold at once: CTAs go through rows with the weights in
// registers, and every thread copies its own pieces of the rows ahead into shared
// memory (cp.async), so loads stay in flight across the two sums of a row; what a thread
// reads it has copied itself, so the ring needs no barrier.  The arithmetic is on
// pairs of floats: issue slots come second to memory.
// row_kernel: one CTA per row, N pieces of VEC elements per thread, T pieces apart (VEC
// = 8 for aligned rows, 1 for layouts nothing else takes).
// flat_kernel: rows without gaps that are not whole 16-byte pieces, in aligned pieces.
// Measured, ring / row: 8,192 x 4,096 bf16 with a gate per channel 44.6 us (6.0 TB/s) /
// 56.9; 8,192 x 2,048 bf16 with a gate per row 28.1 / 32.6; but with an fp32 residual, whose
// rows put half as many bytes again in flight, 40.8 / 30.8 (6.5 TB/s) for 8,192 x 2,048
// and 84.3 / 72.0 for 4,096 x 8,192 without a post-norm.  With one row_kernel takes 33.1 and
// 99.0: at 1,024 threads an SM holds one CTA, which has nothing in flight across a row's
// two sums.
#include "block_ops.cuh"
#include "tc.cuh"

namespace moe {
namespace {

using B = __nv_bfloat16;

template <int VEC>
struct Piece {
  float v[VEC];
};

template <int VEC>
__device__ __forceinline__ void load(const B* p, Piece<VEC>& o) {
  if constexpr (VEC == 8) {
    const uint4 q = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o.v[2 * i] = __uint_as_float(w[i] << 16);
      o.v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  } else {
    o.v[0] = __bfloat162float(*p);
  }
}
template <int VEC>
__device__ __forceinline__ void load(const float* p, Piece<VEC>& o) {
  if constexpr (VEC == 8) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    o.v[0] = a.x, o.v[1] = a.y, o.v[2] = a.z, o.v[3] = a.w;
    o.v[4] = b.x, o.v[5] = b.y, o.v[6] = b.z, o.v[7] = b.w;
  } else {
    o.v[0] = *p;
  }
}
template <int VEC>
__device__ __forceinline__ void store(B* p, const Piece<VEC>& o) {
  if constexpr (VEC == 8) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(o.v[2 * i], o.v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    *p = __float2bfloat16_rn(o.v[0]);
  }
}
template <int VEC>
__device__ __forceinline__ void store(float* p, const Piece<VEC>& o) {
  if constexpr (VEC == 8) {
    *reinterpret_cast<float4*>(p) = make_float4(o.v[0], o.v[1], o.v[2], o.v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(o.v[4], o.v[5], o.v[6], o.v[7]);
  } else {
    *p = o.v[0];
  }
}

// sum over the CTA, the same bits in every thread; `red` is this call's alone
__device__ __forceinline__ float cta_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int warps = blockDim.x >> 5;
  if (warps == 1) return v;
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = (int)(threadIdx.x & 31) < warps ? red[threadIdx.x & 31] : 0.f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// z sigmoid(g) of a bf16 gate.  With n = -g, e^n = 2^(n log2 e); divisor and dividend are a
// quarter of 1 + e^n and of z, below 2^126 for every e^n that fp32 holds, so that the
// reciprocal is a normal number.  n log2 e rounds, an error of up to |g| 2^-24 of the
// result: far below a bf16 residual's own rounding.  EXACT, for an fp32 residual, takes
// e^n = 2^(n hi) e^(n c): hi is the first 16 bits of log2 e, so that n hi is exact, and
// c = 1 - hi ln 2, where 1 + n c leaves 1.5 u at n = 88; every step is within an ulp or two.
// (expf instead: 63.0 us for 8,192 x 4,096 bf16 with a gate per row, 44.7 for 8,192 x 2,048
// fp32, where these take 52.3 and 39.6; EXACT for bf16 too: 55.8.)
template <bool EXACT>
__device__ __forceinline__ float times_sigmoid(float z, float g) {
  constexpr float kLog2e = 1.44269504f, kHi = 47274.f / 32768.f, kC = 4.88849515e-6f;
  float n = -g, e, r;
  if (EXACT) asm("max.NaN.f32 %0, %1, %2;" : "=f"(n) : "f"(n), "f"(-128.f));  // -inf would meet e = 0
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(fmaf(n, EXACT ? kHi : kLog2e, -2.f)));
  if (EXACT) e = fmaf(e, n * kC, e);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(e + 0.25f));
  return 0.25f * z * r;
}

template <int GATE, bool EXACT>
__device__ __forceinline__ float gated(float z, float g) {
  if (GATE == MOE_GATE_LINEAR) return z * g;
  if (GATE == MOE_GATE_SIGMOID) return times_sigmoid<EXACT>(z, g);
  return z;
}

__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   (uint32_t)__cvta_generic_to_shared(dst)),
               "l"(src)
               : "memory");
}

// two floats at a time
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ void unpack(uint4 q, float2 (&o)[4]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
}
__device__ __forceinline__ void store(B* p, const float2 (&o)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __float22bfloat162_rn(o[i]);
    w[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
// D rows in flight per CTA; a slot holds a thread's pieces of h, y and, with a gate
// for each row (GATE), of that.  What multiplies y the same in every row, alpha
// (w_offset + post_w) act(gate), is one fp32 factor per element, made once.
template <int N, int GATE, int D>
__global__ void __launch_bounds__(512, N == 1 ? 2 : 1) ring_kernel(NormArgs a) {
  extern __shared__ uint4 ring[];
  __shared__ float red[2][2][32];
  constexpr int kWords = 2 + (GATE != MOE_GATE_NONE);
  tc::pdl_trigger();
  tc::pdl_wait();
  const int T = blockDim.x, n = a.hidden / 8;
  auto slot = [&](int d, int i, int w) -> uint4* {
    return ring + ((d * N + i) * kWords + w) * T + threadIdx.x;
  };
  auto fetch = [&](long long row, int d) {
    if (row < a.rows) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int at = i * T + (int)threadIdx.x;
        if (at >= n) break;
        copy16(slot(d, i, 0), static_cast<const B*>(a.h) + row * a.h_stride + at * 8);
        if (a.y) copy16(slot(d, i, 1), a.y + row * a.y_stride + at * 8);
        if (GATE != MOE_GATE_NONE) copy16(slot(d, i, 2), a.gate + row * a.gate_stride + at * 8);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int d = 0; d < D - 1; ++d) fetch(blockIdx.x + (long long)d * gridDim.x, d);
  const float2 offset = both(a.w_offset);
  float2 f[N][4];
  uint4 qw[N] = {};
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int at = i * T + (int)threadIdx.x;
#pragma unroll
    for (int j = 0; j < 4; ++j) f[i][j] = both(a.alpha);
    if (at >= n) break;
    float2 w[4];
    if (a.post_w) {
      unpack(reinterpret_cast<const uint4*>(a.post_w)[at], w);
#pragma unroll
      for (int j = 0; j < 4; ++j) f[i][j] = __fmul2_rn(f[i][j], __fadd2_rn(offset, w[j]));
    }
    if (GATE == MOE_GATE_NONE && a.gate) {
      unpack(reinterpret_cast<const uint4*>(a.gate)[at], w);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        f[i][j] = a.gate_kind == MOE_GATE_LINEAR
                      ? __fmul2_rn(f[i][j], w[j])
                      : make_float2(times_sigmoid<true>(f[i][j].x, w[j].x), times_sigmoid<true>(f[i][j].y, w[j].y));
    }
    if (a.pre_w) qw[i] = reinterpret_cast<const uint4*>(a.pre_w)[at];
  }
  const float inv_h = 1.f / (float)a.hidden;
  int d = 0, odd = 0;
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x, odd ^= 1) {
    fetch(row + (long long)(D - 1) * gridDim.x, d == 0 ? D - 1 : d - 1);
    asm volatile("cp.async.wait_group %0;" ::"n"(D - 1) : "memory");
    float2 h[N][4], z[N][4];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const bool in = i * T + (int)threadIdx.x < n;
      const uint4 none = make_uint4(0, 0, 0, 0);
      unpack(in ? *slot(d, i, 0) : none, h[i]);
      unpack(in && a.y ? *slot(d, i, 1) : none, z[i]);
    }
    if (a.y) {
      float2 inv = both(1.f);
      if (a.post_w) {
        float2 s = both(0.f);
#pragma unroll
        for (int i = 0; i < N; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) s = __ffma2_rn(z[i][j], z[i][j], s);
        inv = both(rsqrtf(cta_sum(s.x + s.y, red[odd][0]) * inv_h + a.eps));
      }
#pragma unroll
      for (int i = 0; i < N; ++i) {
        float2 w[4];
        if (GATE != MOE_GATE_NONE && i * T + (int)threadIdx.x < n) unpack(*slot(d, i, 2), w);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          z[i][j] = __fmul2_rn(z[i][j], inv);
          if (GATE != MOE_GATE_NONE)
            z[i][j] = make_float2(gated<GATE, false>(z[i][j].x, w[j].x), gated<GATE, false>(z[i][j].y, w[j].y));
          h[i][j] = __ffma2_rn(z[i][j], f[i][j], h[i][j]);
        }
      }
    }
    d = d + 1 == D ? 0 : d + 1;
    float2 s = both(0.f);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = i * T + (int)threadIdx.x;
      if (at >= n) break;
      if (a.h_out) store(static_cast<B*>(a.h_out) + row * a.ho_stride + at * 8, h[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) s = __ffma2_rn(h[i][j], h[i][j], s);
    }
    if (!a.pre_w) continue;
    const float2 inv = both(rsqrtf(cta_sum(s.x + s.y, red[odd][1]) * inv_h + a.eps));
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = i * T + (int)threadIdx.x;
      if (at >= n) break;
      float2 w[4];
      unpack(qw[i], w);
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = __fmul2_rn(__fmul2_rn(h[i][j], inv), __fadd2_rn(offset, w[j]));
      store(a.x_out + row * a.xo_stride + at * 8, w);
    }
  }
}

template <typename R, int VEC, int N, int GATE>
__global__ void __launch_bounds__(VEC == 1 && N == 8 ? 512 : 1024, VEC == 1 && N == 8 ? 3 : 1)
row_kernel(NormArgs a) {
  __shared__ float red[2][32];
  tc::pdl_trigger();
  tc::pdl_wait();
  const int H = a.hidden, T = blockDim.x;
  const long long b = blockIdx.x;
  const float inv_h = 1.f / (float)H;
  auto at = [&](int i) { return (i * T + (int)threadIdx.x) * VEC; };
  Piece<VEC> h[N], z[N];
  const R* hr = static_cast<const R*>(a.h) + b * a.h_stride;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (at(i) < H) {
      load<VEC>(hr + at(i), h[i]);
      if (a.y) load<VEC>(a.y + b * a.y_stride + at(i), z[i]);
    }
  if (a.y) {
    float inv = 1.f;
    if (a.post_w) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (at(i) < H) {
#pragma unroll
          for (int j = 0; j < VEC; ++j) s = fmaf(z[i].v[j], z[i].v[j], s);
        }
      inv = rsqrtf(cta_sum(s, red[0]) * inv_h + a.eps);
    }
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (at(i) < H) {
        Piece<VEC> w;
        if (a.post_w) {
          load<VEC>(a.post_w + at(i), w);
#pragma unroll
          for (int j = 0; j < VEC; ++j) z[i].v[j] *= inv * (a.w_offset + w.v[j]);
        }
        if (GATE != MOE_GATE_NONE) load<VEC>(a.gate + b * a.gate_stride + at(i), w);
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          h[i].v[j] = fmaf(a.alpha, gated<GATE, sizeof(R) == 4>(z[i].v[j], w.v[j]), h[i].v[j]);
      }
  }
  if (a.h_out) {
    R* o = static_cast<R*>(a.h_out) + b * a.ho_stride;
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (at(i) < H) store<VEC>(o + at(i), h[i]);
  }
  if (!a.pre_w) return;
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (at(i) < H) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) s = fmaf(h[i].v[j], h[i].v[j], s);
    }
  const float inv = rsqrtf(cta_sum(s, red[1]) * inv_h + a.eps);
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (at(i) < H) {
      Piece<VEC> w;
      load<VEC>(a.pre_w + at(i), w);
#pragma unroll
      for (int j = 0; j < VEC; ++j) w.v[j] = h[i].v[j] * inv * (a.w_offset + w.v[j]);
      store<VEC>(a.x_out + b * a.xo_stride + at(i), w);
    }
}

// 8 bf16 that start S elements before the second of two neighbouring words
template <int S>
__device__ __forceinline__ uint4 join(uint4 a, uint4 b) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int k = (8 - S) / 2 + i;
    o[i] = S & 1 ? __funnelshift_r(w[k], w[k + 1 < 8 ? k + 1 : 7], 16) : w[k];
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// Rows without gaps that are not whole 16-byte pieces: the matrices are taken as flat
// arrays in aligned pieces of 8, of which a row's first and last may be shared with
// its neighbours; every array is `off` = row * hidden % 8 elements off the weights,
// which are read as two pieces and shifted.  One piece per thread, 32 registers: a few
// spills cost less than half the threads (8,192 x 4,095 bf16 with a gate 89 us, 107 with
// 44 registers, 126 element by element in row_kernel).
template <typename R, int GATE>
__global__ void __launch_bounds__(1024, 2) flat_kernel(NormArgs a) {
  __shared__ float red[2][32];
  tc::pdl_trigger();
  tc::pdl_wait();
  const int H = a.hidden, tid = threadIdx.x;
  const long long o = (long long)blockIdx.x * H, at = ((o >> 3) + tid) * 8;
  const int off = (int)(o & 7);
  // elements lo .. hi - 1 of this piece are the row's
  const int lo = tid == 0 ? off : 0, hi = (int)min(8LL, max(0LL, o + H - at));
  const bool mine = lo < hi, whole = at + 8 <= (long long)a.rows * H;
  const float inv_h = 1.f / (float)H;
  auto read = [&](auto* p, Piece<8>& v) {
    if (mine && whole) {
      load<8>(p + at, v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v.v[j] = j >= lo && j < hi ? v.v[j] : 0.f;
    } else {  // past the last row there may be no more memory
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        Piece<1> e{{0.f}};
        if (j >= lo && j < hi) load<1>(p + at + j, e);
        v.v[j] = e.v[0];
      }
    }
  };
  auto write = [&](auto* p, const Piece<8>& v) {
    if (lo == 0 && hi == 8) {
      store<8>(p + at, v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const Piece<1> e{{v.v[j]}};
        if (j >= lo && j < hi) store<1>(p + at + j, e);
      }
    }
  };
  // the weights of this piece: elements 8 tid - off ..
  auto weights = [&](const B* p, Piece<8>& v) {
    if (tid > 0 && 8 * tid + 8 <= H) {
      const uint4 hi_w = reinterpret_cast<const uint4*>(p)[tid];
      const uint4 lo_w = off ? reinterpret_cast<const uint4*>(p)[tid - 1] : hi_w;
      uint4 q = hi_w;
      switch (off) {
        case 1: q = join<1>(lo_w, hi_w); break;
        case 2: q = join<2>(lo_w, hi_w); break;
        case 3: q = join<3>(lo_w, hi_w); break;
        case 4: q = join<4>(lo_w, hi_w); break;
        case 5: q = join<5>(lo_w, hi_w); break;
        case 6: q = join<6>(lo_w, hi_w); break;
        case 7: q = join<7>(lo_w, hi_w); break;
      }
      load<8>(reinterpret_cast<const B*>(&q), v);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        Piece<1> e{{0.f}};
        if (j >= lo && j < hi) load<1>(p + 8 * tid - off + j, e);
        v.v[j] = e.v[0];
      }
    }
  };
  Piece<8> h, z, w;
  read(static_cast<const R*>(a.h), h);
  if (a.y) {
    read(a.y, z);
    float inv = 1.f;
    if (a.post_w) {
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) s = fmaf(z.v[j], z.v[j], s);
      inv = rsqrtf(cta_sum(s, red[0]) * inv_h + a.eps);
      weights(a.post_w, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) z.v[j] *= inv * (a.w_offset + w.v[j]);
    }
    if (GATE != MOE_GATE_NONE) {
      if (a.gate_stride) read(a.gate, w);
      else weights(a.gate, w);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) h.v[j] = fmaf(a.alpha, gated<GATE, sizeof(R) == 4>(z.v[j], w.v[j]), h.v[j]);
  }
  if (a.h_out) write(static_cast<R*>(a.h_out), h);
  if (!a.pre_w) return;
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) s = j >= lo && j < hi ? fmaf(h.v[j], h.v[j], s) : s;
  const float inv = rsqrtf(cta_sum(s, red[1]) * inv_h + a.eps);
  weights(a.pre_w, w);
#pragma unroll
  for (int j = 0; j < 8; ++j) w.v[j] = h.v[j] * inv * (a.w_offset + w.v[j]);
  write(a.x_out, w);
}

// flat_kernel's layouts: no gaps, every array 16-byte aligned, at most 1,024 pieces a row
bool flat(const NormArgs& a) {
  const uintptr_t all = reinterpret_cast<uintptr_t>(a.h) | reinterpret_cast<uintptr_t>(a.h_out) |
                        reinterpret_cast<uintptr_t>(a.y) | reinterpret_cast<uintptr_t>(a.post_w) |
                        reinterpret_cast<uintptr_t>(a.gate) | reinterpret_cast<uintptr_t>(a.pre_w) |
                        reinterpret_cast<uintptr_t>(a.x_out);
  const long long H = a.hidden;
  return a.h_stride == H && (!a.y || a.y_stride == H) && (!a.gate_stride || a.gate_stride == H) &&
         (!a.h_out || a.ho_stride == H) && (!a.x_out || a.xo_stride == H) && (all & 15) == 0 && H <= 8176;
}

// every row of every operand starts on a VEC = 8 boundary
template <typename R>
bool vectors(const NormArgs& a) {
  const uintptr_t res = reinterpret_cast<uintptr_t>(a.h) | reinterpret_cast<uintptr_t>(a.h_out);
  const uintptr_t bf = reinterpret_cast<uintptr_t>(a.y) | reinterpret_cast<uintptr_t>(a.post_w) |
                       reinterpret_cast<uintptr_t>(a.gate) | reinterpret_cast<uintptr_t>(a.pre_w) |
                       reinterpret_cast<uintptr_t>(a.x_out);
  const long long strides = a.h_stride | a.y_stride | a.gate_stride | a.ho_stride | a.xo_stride;
  return a.hidden % 8 == 0 && strides % 8 == 0 && ((res | bf) & 15) == 0;
}

template <typename R, int GATE>
cudaError_t launch_rows(const NormArgs& a, cudaStream_t s) {
  auto go = [&](auto kern, int pieces, int per_thread) {
    const int threads = ((pieces + per_thread - 1) / per_thread + 31) / 32 * 32;
    return tc::launch_early(kern, dim3(a.rows), dim3(threads), 0, s, a);
  };
  if (vectors<R>(a))
    return a.hidden <= 8192 ? go(row_kernel<R, 8, 1, GATE>, a.hidden / 8, 1) : go(row_kernel<R, 8, 4, GATE>, a.hidden / 8, 4);
  if (flat(a)) return go(flat_kernel<R, GATE>, a.hidden / 8 + 2, 1);
  if (a.hidden <= 1024) return go(row_kernel<R, 1, 4, GATE>, a.hidden, 4);
  if (a.hidden <= 4096) return go(row_kernel<R, 1, 8, GATE>, a.hidden, 8);
  if (a.hidden <= 8192) return go(row_kernel<R, 1, 16, GATE>, a.hidden, 16);
  return go(row_kernel<R, 1, 32, GATE>, a.hidden, 32);
}

template <int N, int GATE, int D>
cudaError_t launch_ring(const NormArgs& a, int threads, int row_bytes, int sms, cudaStream_t s) {
  auto kern = ring_kernel<N, GATE, D>;
  static tc::Once once;
  const cudaError_t e = tc::raise_smem(once, kern, 131072);
  if (e != cudaSuccess) return e;
  // CTAs an SM holds: by registers (the launch bounds) and shared memory
  const int smem = D * row_bytes, by_smem = 220 * 1024 / (smem + 1536);
  int fit = 512 * (N == 1 ? 2 : 1) / threads;
  fit = fit > by_smem ? by_smem : fit;
  fit = fit > 24 ? 24 : fit < 1 ? 1 : fit;
  const long long grid = (long long)sms * fit;
  return tc::launch_early(kern, dim3((unsigned)(a.rows < grid ? a.rows : grid)), dim3(threads), smem, s, a);
}

template <int GATE>
cudaError_t launch_depth(const NormArgs& a, int threads, int sms, cudaStream_t s) {
  const bool two = a.hidden > 4096;  // pieces per thread
  const int row = threads * (two ? 2 : 1) * 16 * (2 + (GATE != MOE_GATE_NONE));
  // four rows in flight where two CTAs of them fit an SM
  if (4 * row <= 108 * 1024)
    return two ? launch_ring<2, GATE, 4>(a, threads, row, sms, s) : launch_ring<1, GATE, 4>(a, threads, row, sms, s);
  return launch_ring<2, GATE, 2>(a, threads, row, sms, s);
}

template <typename R, int GATE>
cudaError_t launch(const NormArgs& a, cudaStream_t s) {
  if constexpr (sizeof(R) == 2) {
    tc::DeviceInfo dev;
    const cudaError_t e = tc::device_info(&dev);
    if (e != cudaSuccess) return e;
    const int n = a.hidden / 8, per = n <= 512 ? 1 : 2, threads = ((n + per - 1) / per + 31) / 32 * 32;
    if (vectors<R>(a) && n <= 1024 && a.rows > (long long)dev.sms * (1024 / threads)) {
      if (GATE == MOE_GATE_NONE || a.gate_stride == 0) return launch_depth<MOE_GATE_NONE>(a, threads, dev.sms, s);
      return launch_depth<GATE>(a, threads, dev.sms, s);
    }
  }
  return launch_rows<R, GATE>(a, s);
}

template <typename R>
cudaError_t by_gate(const NormArgs& a, cudaStream_t s) {
  if (a.gate_kind == MOE_GATE_LINEAR) return launch<R, MOE_GATE_LINEAR>(a, s);
  if (a.gate_kind == MOE_GATE_SIGMOID) return launch<R, MOE_GATE_SIGMOID>(a, s);
  return launch<R, MOE_GATE_NONE>(a, s);
}

}  // namespace

cudaError_t launch_block_norm(const NormArgs& a, int res_dtype, cudaStream_t s) {
  return res_dtype == MOE_T_F32 ? by_gate<float>(a, s) : by_gate<B>(a, s);
}

}  // namespace moe

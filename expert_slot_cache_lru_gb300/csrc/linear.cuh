// linear.cuh -- what the bf16 products share: activations, the end of a result, and
// the walk over the tiles of ragged groups.
#pragma once

#include "block_ops.cuh"

namespace moe {
namespace lin {

constexpr unsigned kAll = 0xffffffffu;

// e^-|z| over a divisor of 1 .. 2, where __fdividef has 2 ulp; NaN for a NaN
__device__ __forceinline__ float sigmoid(float z) {
  const float e = expf(-fabsf(z));
  return __fdividef(z < 0.f ? e : 1.f, 1.f + e);
}
// z Phi(z) by the upper tail Q(a) = e^(-a^2 / 2) R(a), a = |z|: no cancellation in Phi's lower tail.  R is the
// smooth scaled tail erfcx(a / sqrt 2) / 2, here t times a polynomial of degree 8 in t = 1 / (1 + 0.35 a), fitted for least
// relative error over 0 .. 16 (2^-24); the exponent's rounding a^2 - fl(a^2) is put back.  All of it is at most 7.8 2^-24
// off, over 6 million fp32 z of -12.5 .. 6.
// 8,192 x 8,192 x 512 with a residual 232 us, by normcdff (67 cycles a lane) 291.
__device__ __forceinline__ float gelu(float z) {
  const float a = fminf(fabsf(z), 16.f);  // Q(16) is below fp32; a NaN comes back with z
  const float d = fmaf(0.35f, a, 1.f), t0 = __fdividef(1.f, d), t = fmaf(t0, fmaf(-d, t0, 1.f), t0);
  float r = -0.029164928942918777f;
  r = fmaf(r, t, 0.1440657675266266f);
  r = fmaf(r, t, -0.25591233372688293f);
  r = fmaf(r, t, 0.1594051569700241f);
  r = fmaf(r, t, -0.023272467777132988f);
  r = fmaf(r, t, 0.10557854920625687f);
  r = fmaf(r, t, 0.11981452256441116f);
  r = fmaf(r, t, 0.1398644745349884f);
  r = fmaf(r, t, 0.13962124288082123f);
  const float s = a * a, lost = fmaf(a, a, -s);
  const float q = r * t * expf(-0.5f * s) * fmaf(-0.5f, lost, 1.f);
  return z * (z < 0.f ? q : 1.f - q);
}
template <int ACT>
__device__ __forceinline__ float act1(float z) {
  if constexpr (ACT == MOE_ACT_SILU) return z * sigmoid(z);
  if constexpr (ACT == MOE_ACT_GELU) return gelu(z);
  // (1 + tanh u) / 2 is the sigmoid of 2 u, which does not cancel
  if constexpr (ACT == MOE_ACT_GELU_TANH) return z * sigmoid(1.5957691216f * fmaf(0.044715f * z, z * z, z));
  if constexpr (ACT == MOE_ACT_RELU) return z < 0.f ? 0.f : z;
  return z;
}
template <int A>
struct Act {
  __device__ __forceinline__ float operator()(float z) const { return act1<A>(z); }
};
// f with the activation as its argument: one branch around a loop over many values
template <typename F>
__device__ __forceinline__ void with_act(int act, F f) {
  if (act == MOE_ACT_SILU) f(Act<MOE_ACT_SILU>{});
  else if (act == MOE_ACT_GELU) f(Act<MOE_ACT_GELU>{});
  else if (act == MOE_ACT_GELU_TANH) f(Act<MOE_ACT_GELU_TANH>{});
  else if (act == MOE_ACT_RELU) f(Act<MOE_ACT_RELU>{});
  else f(Act<MOE_ACT_NONE>{});
}

__device__ __forceinline__ float load_res(const Linear& l, long long at) {
  return l.f32 ? static_cast<const float*>(l.res)[at]
               : __bfloat162float(static_cast<const __nv_bfloat16*>(l.res)[at]);
}
__device__ __forceinline__ void store_out(const Linear& l, long long at, float v) {
  if (l.f32) static_cast<float*>(l.out)[at] = v;
  else static_cast<__nv_bfloat16*>(l.out)[at] = __float2bfloat16_rn(v);
}
// res + alpha * y at (row, n)
__device__ __forceinline__ void finish(const Linear& l, long long row, long long n, float y) {
  const float v = l.res ? fmaf(l.alpha, y, load_res(l, row * l.res_stride + n)) : l.alpha * y;
  store_out(l, row * l.out_stride + n, v);
}

// The row of x behind an entry of the order, or -1 where there is none: r / per_row by a product (per_mul and
// per_shift from division_of).
__device__ __forceinline__ int row_of(const Linear& l, int r) {
  const int b = (int)((__umulhi(l.per_mul, (unsigned)r) + (unsigned)r) >> l.per_shift);
  return r >= 0 && b < l.x_rows ? b : -1;
}
// ... behind place p
__device__ __forceinline__ int source_row(const Linear& l, int p) { return l.order ? row_of(l, l.order[p]) : p; }

// Factor and shift with (umulhi(mul, r) + r) >> shift == r / d for 0 <= r < 2^31: with 2^shift >= d the factor is
// 2^32 (2^shift - d) / d + 1, rounded down, so that mul + 2^32 is 2^(32 + shift) / d to an excess of at most 1,
// which r < 2^31 times makes less than a step of the quotient.
inline void division_of(int d, unsigned& mul, int& shift) {
  shift = 0;
  while ((1ll << shift) < d) ++shift;
  mul = (unsigned)((((1ull << shift) - d) << 32) / d + 1);
}

// Tiles of ragged groups in order, for a warp that asks for rising tile numbers.  A
// group of R rows has ceil(R / 2^shift) tiles of equal size (up to a multiple of gran) by `tn`
// tiles of n; the tiles of n run fastest, in strips of 8, so that tiles that run at the
// same time share operands in L2.  128 groups are looked at together: each lane counts the
// tiles of four, and a scan over the lanes finds the one a tile is in.  The next 128 groups' offsets
// are loaded ahead.
struct Tile {
  int group, row, rows, n;  // rows: of this tile; n: which tile of n
};
struct Walk {
  const int32_t* offsets;
  int groups, total_rows, shift, gran, tn;  // tiles of up to 1 << shift rows
  int g0;         // first group of this chunk
  int reach;      // where the groups so far end
  int base, end;  // tile numbers of this chunk
  int lo[4], hi[4], ahead[5], incl;
  int dense_tiles, dense_width;  // of tokens, where there are no groups

  __device__ __forceinline__ void load(int g) {  // into `ahead`, lane's four groups of a chunk
#pragma unroll
    for (int i = 0; i < 5; ++i) {
      const int at = g + 4 * (int)(threadIdx.x & 31) + i;
      ahead[i] = offsets ? offsets[min(at, groups)] : (at == 0 ? 0 : total_rows);
    }
  }
  __device__ __forceinline__ int parts(int rows) const {  // rows up to 2^31 - 1
    return (int)(((unsigned)rows + (1u << shift) - 1) >> shift);
  }
  __device__ __forceinline__ int tiles(int i) const { return parts(hi[i] - lo[i]) * tn; }
  __device__ __forceinline__ void take() {  // the chunk from `ahead`
    // offsets within 0 .. total_rows; a group starts no earlier than those before it end, so that offsets
    // that do not ascend make no more tiles than there can be
    int most = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo[i] = min(max(ahead[i], 0), total_rows);
      hi[i] = min(max(ahead[i + 1], 0), total_rows);
      most = max(most, max(lo[i], hi[i]));
    }
    int upto = most;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kAll, upto, o);
      if ((int)(threadIdx.x & 31) >= o) upto = max(upto, v);
    }
    const int before = __shfl_up_sync(kAll, upto, 1);
    int from = (threadIdx.x & 31) ? max(reach, before) : reach, sum = 0;
    reach = max(reach, __shfl_sync(kAll, upto, 31));
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo[i] = max(lo[i], from);
      from = hi[i] = max(hi[i], lo[i]);
      sum += tiles(i);
    }
    incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(kAll, incl, o);
      if ((int)(threadIdx.x & 31) >= o) incl += v;
    }
    end = base + __shfl_sync(kAll, incl, 31);
  }
  // tiles, width: of a dense product (0: as for a group)
  __device__ __forceinline__ void start(const Linear& l, int shift_, int gran_, int tn_, int tiles = 0, int width = 0) {
    offsets = l.offsets;
    dense_tiles = tiles;
    dense_width = width;
    groups = l.groups;
    total_rows = l.rows;
    shift = shift_;
    gran = gran_;
    tn = tn_;
    if (dense_tiles) return;
    g0 = base = reach = 0;
    load(0);
    take();
    load(128);
  }
  // tile r of T by tn tiles of `width` rows from lo to hi
  __device__ __forceinline__ void place(int r, int T, int width, int lo_, int hi_, Tile& out) const {
    const int per = 8 * T, strip = r / per, in = r - strip * per, w = min(8, tn - strip * 8);
    out.n = strip * 8 + in % w;
    out.row = lo_ + in / w * width;
    out.rows = min(width, hi_ - out.row);
  }
  // false where tile t is past the last
  __device__ __forceinline__ bool seek(int t, Tile& out) {
    if (dense_tiles) {
      if (t >= dense_tiles * tn) return false;
      out.group = 0;
      place(t, dense_tiles, dense_width, 0, total_rows, out);
      return true;
    }
    while (t >= end) {
      g0 += 128;
      if (g0 >= groups) return false;
      base = end;
      take();
      load(g0 + 128);
    }
    int r = t - base;
    const int lane = __ffs(__ballot_sync(kAll, incl > r)) - 1;
    int mine = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) mine += tiles(i);
    r -= __shfl_sync(kAll, incl - mine, lane);
    int l0 = 0, h0 = 0, g = 0;
    bool found = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int a = __shfl_sync(kAll, lo[i], lane), b = __shfl_sync(kAll, hi[i], lane);
      const int n = parts(b - a) * tn;
      if (!found && r < n) {
        found = true;
        l0 = a;
        h0 = b;
        g = g0 + 4 * lane + i;
      }
      if (!found) r -= n;
    }
    if (!found) return false;
    const int R = h0 - l0, T = parts(R);
    out.group = g;
    place(r, T, ((R - 1) / T + gran) / gran * gran, l0, h0, out);  // ceil(R / T), up to a multiple of gran
    return true;
  }
};

// Most tiles there can be, for a grid.
inline long long most_tiles(const Linear& l, int shift, long long tn) {
  const long long part = l.rows < l.groups ? l.rows : l.groups;
  return (((long long)l.rows >> shift) + part) * tn;
}

}  // namespace lin
}  // namespace moe

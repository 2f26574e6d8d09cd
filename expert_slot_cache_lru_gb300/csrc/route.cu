// route.cu -- the router: logits, scores, grouped choice and weights
// (formulas in moe_cache.h).
//
// Selection: one warp owns a row.  Each of the G groups takes 32 / G lanes, and
// a lane every (32 / G)-th expert of its group, up to 32 of them in registers: loads are
// coalesced, and the groups' scores are one reduction over 32 / G lanes for all
// groups at once.  Choices are compared as unsigned integers in the order of
// the floats (0 = masked), which makes a pick two warp reductions: the largest
// key, then the lowest id among its holders.  Group counts that do not divide 32 and more
// than 32 experts per lane take one CTA per row with the keys in shared memory.
//
// Logits: up to kDotRows rows are dot products, one CTA per expert (its router row
// read once for all rows; with the selection 6.8 us for 8 rows x 2,048 x 256 and 9.9
// for 16, on the tensor cores 9.1 for either); more rows are a product on the tensor cores
// (tile_gemm.cuh), whose operands must start on 16 bytes; other layouts take tile_dot.cuh.
// The selection is a second launch that starts while the logits are computed and waits for
// them: 950 warp instructions a row for 8 of 256 in 8 groups, 10.8 us for 8,192 rows.
#include "block_ops.cuh"
#include "tile_dot.cuh"
#include "tile_gemm.cuh"

namespace moe {
namespace {

constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ float load_f(const float* p) { return *p; }
__device__ __forceinline__ float load_f(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// order of floats as unsigned integers; NaN and -inf (masked) are 0
__device__ __forceinline__ uint32_t choice_key(float c) {
  if (!(c > -INFINITY)) return 0u;
  const uint32_t u = __float_as_uint(c + 0.f);  // -0 and +0 tie
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
// The key of a group's two largest values; a sum below the type's lowest value is that
// value, since the group has unmasked experts.
__device__ __forceinline__ uint32_t sum_key(float v1, float v2) {
  return choice_key(fmaxf(v1 + v2, -3.40282347e38f));
}

// Score numerators: the sigmoid, or softmax's exp(z - max).  Scores far below the largest
// can decide (a bias or groups leave the largest out, shares are renormalised), so the
// exponential is expf, 2 ulp; __expf's error grows with its argument, 60 u at e^-60 (and
// saves 0.4 us of 16.6 for 600 rows of 1,024 experts, 0.5 of 32.6 for 8,192 of 256).  The
// sigmoid's divisor lies in 1 .. 2, where __fdividef has 2 ulp; 1 + e^-z would leave its
// range while the quotient still is a number.
__device__ __forceinline__ float sigmoid(float z) {  // NaN for a NaN
  const float e = expf(-fabsf(z));
  return __fdividef(z < 0.f ? e : 1.f, 1.f + e);
}
__device__ __forceinline__ float softmax_term(float z, float zmax) {
  if (!(z > -INFINITY)) return 0.f;
  if (zmax == INFINITY) return z == INFINITY ? 1.f : 0.f;
  return expf(z - zmax);
}
__device__ __forceinline__ float raw_score(float z, bool softmax, float zmax) {
  if (softmax) return softmax_term(z, zmax);
  return z > -INFINITY ? sigmoid(z) : 0.f;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}

// writes a row's picks: lane r < k holds pick r (id -1: none) and its logit.  A softmax's
// renormalised weights are taken from the picks alone, by their largest logit: shares of
// scores that fp32 does not hold.
__device__ __forceinline__ void write_row(const RouteArgs& a, long long b, int lane, int id, float z,
                                          bool softmax, float zmax, float inv) {
  const bool picked = lane < a.k && id >= 0;
  if (softmax && a.renorm && zmax < INFINITY) {
    zmax = warp_max(picked ? z : -INFINITY);
    inv = 1.f;
  }
  float w = picked ? raw_score(z, softmax, zmax) * inv : 0.f;
  if (a.renorm) {
    const float t = warp_sum(w);
    w = t > 0.f ? w / t : 0.f;
  }
  if (lane < a.k) {
    a.ids[b * a.k + lane] = id;
    a.w[b * a.k + lane] = w * a.scale;
  }
}

// a lane's two largest keys and their places j, the lower place first among equals
struct Top2 {
  uint32_t k1, k2;
  int i1, i2;
};
template <int EL>
__device__ __forceinline__ Top2 top2(const uint32_t (&key)[EL], uint32_t gone) {
  Top2 t{0u, 0u, 0, 0};
#pragma unroll
  for (int j = 0; j < EL; ++j) {
    const uint32_t k = (gone >> j) & 1 ? 0u : key[j];
    const bool first = k > t.k1, second = k > t.k2;
    t.i2 = first ? t.i1 : second ? j : t.i2;
    t.k2 = first ? t.k1 : second ? k : t.k2;
    t.i1 = first ? j : t.i1;
    t.k1 = first ? k : t.k1;
  }
  return t;
}

// `shift`: log2 of the lanes per group; gs: experts per group.  Each lane keeps its two
// best keys, which serve its first two picks and its group's score; a lane that is
// picked from twice looks through its keys again.  A pick's score is made again from
// its logit, by the lane that writes it, so that no scores move with the picks.
template <int EL, bool BIAS, typename T>
__global__ void __launch_bounds__(128) select_warp_kernel(RouteArgs a, int shift, int gs) {
  tc::pdl_trigger();
  const long long b = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (b >= a.rows) return;
  const int lane = threadIdx.x & 31, lanes = 1 << shift, group = lane >> shift;
  // lane's experts: first + j * lanes, below end
  const int first = group * gs + (lane & (lanes - 1)), end = (group + 1) * gs;
  const T* zr = static_cast<const T*>(a.logits) + b * a.stride;
  const bool softmax = a.score == MOE_SCORE_SOFTMAX;
  tc::pdl_wait();
  float s[EL];
  uint32_t key[EL];
  float mx = -INFINITY, inv = 1.f;
  float b_e[BIAS ? EL : 1];  // loaded before the first use: behind a condition they came one by one
  if (BIAS) {
#pragma unroll
    for (int j = 0; j < EL; ++j)
      b_e[j] = first + (j << shift) < end ? a.bias[first + (j << shift)] : 0.f;
  }
#pragma unroll
  for (int j = 0; j < EL; ++j) {
    s[j] = first + (j << shift) < end ? load_f(zr + first + (j << shift)) : -INFINITY;
    mx = fmaxf(mx, s[j]);  // fmaxf drops NaN
  }
#pragma unroll
  for (int j = 0; j < EL; ++j)  // without a bias the logits rank
    key[j] = BIAS ? s[j] > -INFINITY : choice_key(s[j]);
  if (softmax) mx = warp_max(mx);
  if (softmax) {
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < EL; ++j) sum += s[j] = softmax_term(s[j], mx);
    sum = warp_sum(sum);
    inv = sum > 0.f ? 1.f / sum : 0.f;
  } else if (BIAS) {
#pragma unroll
    for (int j = 0; j < EL; ++j) s[j] = sigmoid(s[j]);  // a masked expert has key 0
  }
  if (BIAS) {
#pragma unroll
    for (int j = 0; j < EL; ++j) {
      const uint32_t c = choice_key(fmaf(s[j], inv, b_e[j]));
      key[j] = key[j] ? c : 0u;
    }
  }
  Top2 t = top2(key, 0u);
  if (a.groups > 1) {
    uint32_t k1 = t.k1, k2 = t.k2;  // the group's two largest choices
    for (int o = lanes >> 1; o > 0; o >>= 1) {
      const uint32_t q1 = __shfl_xor_sync(kAll, k1, o), q2 = __shfl_xor_sync(kAll, k2, o);
      k2 = max(min(k1, q1), max(k2, q2));
      k1 = max(k1, q1);
    }
    uint32_t mine = k1;
    if (a.group_top == 2 && k1) {  // their sum, or of their scores
      float v1 = key_value(k1), v2 = k2 ? key_value(k2) : 0.f;
      if (!BIAS) {
        v1 = raw_score(v1, softmax, mx) * inv;
        v2 = k2 ? raw_score(v2, softmax, mx) * inv : 0.f;
      }
      mine = sum_key(v1, v2);
    }
    int rank = 0;  // groups ahead of this one
    for (int g = 0; g < a.groups; ++g) {
      const uint32_t other = __shfl_sync(kAll, mine, g << shift);
      rank += other > mine || (other == mine && g < group);
    }
    if (rank >= a.topk_groups || !mine) t.k1 = t.k2 = 0u;
  }
  int my_id = -1, left = 2;  // left: best keys at hand
  uint32_t gone = 0u;        // places picked from
  for (int r = 0; r < a.k; ++r) {
    const uint32_t best = __reduce_max_sync(kAll, t.k1);
    if (!best) break;
    const int cand = t.k1 == best ? first + (t.i1 << shift) : 0x7fffffff;
    const int id = __reduce_min_sync(kAll, cand);  // the lowest of its holders
    if (cand == id) {
      gone |= 1u << t.i1;
      t.k1 = t.k2;
      t.i1 = t.i2;
      t.k2 = 0u;
      --left;
    }
    if (__any_sync(kAll, left == 0)) {
      const Top2 again = top2(key, gone);
      if (left == 0) {
        t = again;
        left = 2;
      }
    }
    if (lane == r) my_id = id;
  }
  write_row(a, b, lane, my_id, my_id < 0 ? 0.f : load_f(zr + my_id), softmax, mx, inv);
}

constexpr int kBigThreads = 256;

struct BigSmem {
  float red[kBigThreads / 32];
  uint32_t key[kBigThreads / 32];
  unsigned id[kBigThreads / 32];
  uint32_t gk[64];
  unsigned long long keep;
  int pick[32];
};

// one CTA per row, keys and scores in shared memory
template <typename T>
__global__ void __launch_bounds__(kBigThreads) select_cta_kernel(RouteArgs a) {
  extern __shared__ uint32_t dyn[];
  __shared__ BigSmem sm;
  uint32_t* key = dyn;
  float* s = reinterpret_cast<float*>(dyn + a.E);
  const long long b = blockIdx.x;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const T* zr = static_cast<const T*>(a.logits) + b * a.stride;
  const bool softmax = a.score == MOE_SCORE_SOFTMAX;
  tc::pdl_trigger();
  tc::pdl_wait();
  float mx = -INFINITY;
  for (int e = threadIdx.x; e < a.E; e += kBigThreads) mx = fmaxf(mx, load_f(zr + e));
  mx = warp_max(mx);
  if (lane == 0) sm.red[warp] = mx;
  __syncthreads();
  for (int i = 0; i < kBigThreads / 32; ++i) mx = fmaxf(mx, sm.red[i]);
  __syncthreads();
  float sum = 0.f;
  if (softmax)
    for (int e = threadIdx.x; e < a.E; e += kBigThreads) sum += softmax_term(load_f(zr + e), mx);
  sum = warp_sum(sum);
  if (lane == 0) sm.red[warp] = sum;
  __syncthreads();
  sum = 0.f;
  for (int i = 0; i < kBigThreads / 32; ++i) sum += sm.red[i];
  const float inv = !softmax ? 1.f : sum > 0.f ? 1.f / sum : 0.f;
  for (int e = threadIdx.x; e < a.E; e += kBigThreads) {
    const float z = load_f(zr + e);
    const float sc = raw_score(z, softmax, mx) * inv;
    s[e] = sc;
    key[e] = choice_key(a.bias ? (z > -INFINITY ? sc + a.bias[e] : -INFINITY) : z);
  }
  __syncthreads();
  if (a.groups > 1) {
    const int gs = a.E / a.groups;
    for (int g = warp; g < a.groups; g += kBigThreads / 32) {
      uint32_t k1 = 0u, k2 = 0u;
      float s1 = 0.f, s2 = 0.f;
      for (int e = g * gs + lane; e < (g + 1) * gs; e += 32)
        if (key[e]) {
          k2 = max(k2, min(k1, key[e]));
          k1 = max(k1, key[e]);
          s2 = fmaxf(s2, fminf(s1, s[e]));
          s1 = fmaxf(s1, s[e]);
        }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const uint32_t q1 = __shfl_xor_sync(kAll, k1, o), q2 = __shfl_xor_sync(kAll, k2, o);
        const float t1 = __shfl_xor_sync(kAll, s1, o), t2 = __shfl_xor_sync(kAll, s2, o);
        k2 = max(min(k1, q1), max(k2, q2));
        k1 = max(k1, q1);
        s2 = fmaxf(fminf(s1, t1), fmaxf(s2, t2));
        s1 = fmaxf(s1, t1);
      }
      uint32_t sc = k1;
      if (a.group_top == 2 && k1)
        sc = a.bias ? sum_key(key_value(k1), k2 ? key_value(k2) : 0.f) : sum_key(s1, s2);
      if (lane == 0) sm.gk[g] = sc;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      unsigned long long keep = 0;
      for (int t = 0; t < a.topk_groups; ++t) {
        int at = -1;
        for (int g = 0; g < a.groups; ++g)
          if (sm.gk[g] && (at < 0 || sm.gk[g] > sm.gk[at])) at = g;
        if (at < 0) break;
        keep |= 1ull << at;
        sm.gk[at] = 0u;
      }
      sm.keep = keep;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += kBigThreads)
      if (!((sm.keep >> (e / gs)) & 1)) key[e] = 0u;
    __syncthreads();
  }
  if (threadIdx.x < 32) sm.pick[threadIdx.x] = -1;
  for (int r = 0; r < a.k; ++r) {
    uint32_t top = 0u;
    unsigned at = 0xffffffffu;
    for (int e = threadIdx.x; e < a.E; e += kBigThreads)
      if (key[e] > top) {
        top = key[e];
        at = e;
      }
    const uint32_t wb = __reduce_max_sync(kAll, top);
    const unsigned wi = __reduce_min_sync(kAll, top == wb && wb ? at : 0xffffffffu);
    if (lane == 0) {
      sm.key[warp] = wb;
      sm.id[warp] = wi;
    }
    __syncthreads();
    uint32_t best = 0u;
    unsigned id = 0xffffffffu;
    for (int i = 0; i < kBigThreads / 32; ++i)
      if (sm.key[i] > best || (sm.key[i] == best && sm.id[i] < id)) {
        best = sm.key[i];
        id = sm.id[i];
      }
    if (best && threadIdx.x == 0) {
      sm.pick[r] = (int)id;
      key[id] = 0u;
    }
    __syncthreads();
    if (!best) break;
  }
  if (warp == 0) {
    const int id = sm.pick[lane];
    write_row(a, b, lane, id, id < 0 ? 0.f : load_f(zr + id), softmax, mx, inv);
  }
}

template <typename T>
cudaError_t select(const RouteArgs& a, cudaStream_t s) {
  const int gs = a.E / a.groups;
  int shift = 5;  // lanes per group: 32 / groups
  while (shift > 0 && a.groups << shift > 32) --shift;
  const int per = a.groups << shift == 32 ? (gs + (1 << shift) - 1) >> shift : 33;
  auto go = [&](auto kern) {
    return tc::launch_early(kern, dim3((unsigned)((a.rows + 3LL) / 4)), dim3(128), 0, s, a, shift, gs);
  };
  if (per <= 1) return a.bias ? go(select_warp_kernel<1, true, T>) : go(select_warp_kernel<1, false, T>);
  if (per <= 2) return a.bias ? go(select_warp_kernel<2, true, T>) : go(select_warp_kernel<2, false, T>);
  if (per <= 4) return a.bias ? go(select_warp_kernel<4, true, T>) : go(select_warp_kernel<4, false, T>);
  if (per <= 8) return a.bias ? go(select_warp_kernel<8, true, T>) : go(select_warp_kernel<8, false, T>);
  if (per <= 16) return a.bias ? go(select_warp_kernel<16, true, T>) : go(select_warp_kernel<16, false, T>);
  if (per <= 32) return a.bias ? go(select_warp_kernel<32, true, T>) : go(select_warp_kernel<32, false, T>);
  static tc::Once once;
  const cudaError_t e = tc::raise_smem(once, select_cta_kernel<T>, 16384 * 8);
  if (e != cudaSuccess) return e;
  return tc::launch_early(select_cta_kernel<T>, dim3((unsigned)a.rows), dim3(kBigThreads), (size_t)a.E * 8, s, a);
}

constexpr int kDotRows = 8, kDotWarps = 4;

// z[b][e] for R rows: CTA e, its warps over pieces of 8 elements of K
template <int R>
__global__ void __launch_bounds__(32 * kDotWarps)
dot_kernel(const __nv_bfloat16* x, long long x_stride, const __nv_bfloat16* router, int rows,
           int hidden, int E, float* z) {
  __shared__ float red[kDotWarps][R];
  tc::pdl_trigger();
  tc::pdl_wait();
  const int e = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint4* w = reinterpret_cast<const uint4*>(router + (size_t)e * hidden);
  float acc[R] = {};
#pragma unroll 2
  for (int i = threadIdx.x; i < hidden / 8; i += 32 * kDotWarps) {
    const uint4 wq = w[i];
    const uint32_t wv[4] = {wq.x, wq.y, wq.z, wq.w};
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (r >= rows) break;
      const uint4 xq = reinterpret_cast<const uint4*>(x + r * x_stride)[i];
      const uint32_t xv[4] = {xq.x, xq.y, xq.z, xq.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc[r] = fmaf(__uint_as_float(wv[j] << 16), __uint_as_float(xv[j] << 16), acc[r]);
        acc[r] = fmaf(__uint_as_float(wv[j] & 0xffff0000u), __uint_as_float(xv[j] & 0xffff0000u), acc[r]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const float v = warp_sum(acc[r]);
    if (lane == 0) red[warp][r] = v;
  }
  __syncthreads();
  if (threadIdx.x < R && (int)threadIdx.x < rows) {
    float v = 0.f;
    for (int i = 0; i < kDotWarps; ++i) v += red[i][threadIdx.x];
    z[(size_t)threadIdx.x * E + e] = v;
  }
}

struct Bf16Rows {
  const __nv_bfloat16* p;
  long long stride;
  __device__ float operator()(int r, int k) const { return __bfloat162float(p[r * stride + k]); }
};
struct StoreF32 {
  float* p;
  long long stride;
  __device__ void operator()(int m, int n, float v) const { p[m * stride + n] = v; }
};

}  // namespace

cudaError_t launch_route_select(const RouteArgs& a, int dtype, cudaStream_t s) {
  return dtype == MOE_T_F32 ? select<float>(a, s) : select<__nv_bfloat16>(a, s);
}

cudaError_t launch_route_logits(const __nv_bfloat16* x, long long x_stride,
                                const __nv_bfloat16* router, int rows, int hidden, int E, float* z,
                                unsigned long long* status, cudaStream_t s) {
  const bool whole = hidden % 8 == 0 && x_stride % 8 == 0 &&
                     ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(router)) & 15) == 0;
  if (whole && rows <= kDotRows) {
    auto go = [&](auto kern) {
      return tc::launch_early(kern, dim3(E), dim3(32 * kDotWarps), 0, s, x, x_stride, router, rows, hidden, E, z);
    };
    return rows == 1 ? go(dot_kernel<1>) : rows <= 4 ? go(dot_kernel<4>) : go(dot_kernel<kDotRows>);
  }
  if (whole) {
    tc::DeviceInfo d;
    const cudaError_t e = tc::device_info(&d);
    if (e != cudaSuccess) return e;
    tg::Problem p{};
    p.p = x;
    p.q = router;
    p.p_stride = x_stride * 2;
    p.q_stride = (long long)hidden * 2;
    p.p_rows = rows;
    p.q_rows = E;
    p.k = hidden;
    p.out = z;
    p.out_stride = E;
    p.f32 = true;
    p.status = status;
    const long long c64 = tg::cycles<tg::kBf16, 64, 1>(rows, E, hidden, d.sms),
                    c128 = tg::cycles<tg::kBf16, 128, 1>(rows, E, hidden, d.sms),
                    c256 = tg::cycles<tg::kBf16, 256, 2>(rows, E, hidden, d.sms);
    if (c256 <= c128 && c256 <= c64) return tg::launch<tg::kBf16, 256, 2, false>(p, d.sms, s);
    if (c128 <= c64) return tg::launch<tg::kBf16, 128, 1, false>(p, d.sms, s);
    return tg::launch<tg::kBf16, 64, 1, false>(p, d.sms, s);
  }
  // rows in slices that keep the grid's y within 65,535
  for (long long r0 = 0; r0 < rows; r0 += 65535 * 64) {
    const int n = (int)(rows - r0 < 65535 * 64 ? rows - r0 : 65535 * 64);
    tile_dot_kernel<<<dim3((E + 63) / 64, (n + 63) / 64), 256, 0, s>>>(
        Bf16Rows{x + r0 * x_stride, x_stride}, Bf16Rows{router, hidden},
        StoreF32{z + r0 * E, E}, n, E, hidden);
  }
  return cudaGetLastError();
}

}  // namespace moe

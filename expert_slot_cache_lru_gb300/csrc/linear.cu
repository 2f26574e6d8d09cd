// linear.cu -- the bf16 products (formulas in moe_cache.h): which kernel takes a
// call, the dot products of a few rows, and the tiles for operands of any layout.
//
// A few rows are bound by the weights' bytes: a CTA takes a few rows of weights, its warps a slice of K each, 16 bytes
// a lane and load, all loads of a slice in flight together and x in registers beside them.  Grouped, a place is a
// row of its own: its group is looked up by the whole block at once.  Three to 16 rows take the warps' own MMAs, straight
// from registers: the weights' bytes bound them too, and a tile of the large kernel has its pipeline to fill first.
//
// Layouts the large kernel's copies cannot address (rows that are no whole 16-byte pieces, gated widths that are no
// multiple of 16) take tiles of the warps' MMAs too, bound by loads of two bytes a lane in the eight warps that an SM's
// registers hold (8,192 x 8,192 x 4,097: 4.9 ms; in one truncating chain of K 4.6).
#include "linear.cuh"
#include "tc.cuh"

namespace moe {
namespace {

using namespace lin;

constexpr int kDotThreads = 128, kDotRows = 2;
// CTAs an SM, which bound the registers.  Eight, 64 registers (4,096 x 4,096: 7.4 us, with 77 8.0); seven, 72, for a row with a
// gate, which spills with 64 (8 / 24 places over 256 of 2 x 512 x 2,048: 7.7 / 18.7 us, of eight CTAs 8.1 / 19.4, of six 9.0 /
// 19.0; one row of 2 x 1,024 x 4,096 5.0, 5.4 and 4.6), but not as 16 warps (2 x 512 x 8,192: 4.8 us, with more registers 6.4).
template <int R, bool GATED, int THREADS>
constexpr int kDotCtas = R == 1 && GATED && THREADS == kDotThreads ? 7 : 8 * kDotThreads / THREADS;
constexpr int kStreamRows = 16;
// Rows of weights of a CTA's part and 256-element pieces of K of a warp, for R rows of x: the best of
// 4 and 8 and of 1, 2 and 4 at 4,096 x 4,096 (8.1 and 7.9 us; with more in flight per thread and fewer threads 9
// to 13).
template <int R>
struct Dots {
  static constexpr int NB = 4, U = R == 1 ? 2 : 1;
};

// c += a b^T over 16 of K for 16 rows of a and 8 of b (fp32 += bf16 x bf16).  Lane 4 g + t has rows g and g + 8 of a and
// row g of b, of each the places 2 t, 2 t + 1 and 2 t + 8, 2 t + 9 of K; of c columns 2 t, 2 t + 1.
__device__ __forceinline__ void mma_16x8(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Operands of any layout: tiles of 128 rows x 128 rows of weights (gated: 64 results, their gate and up rows in turns of
// eight, which puts a result's halves into one lane), 32 of K at a time, loaded an element a lane (the next 32 into
// registers while these are multiplied) and from shared memory into the warps' MMAs, 32 x 64 a warp.  The MMAs truncate
// their additions, so each 16 of K is a sum of its own, added to the others in fp32, rounded to nearest.
constexpr int kPitch = 40;  // elements; rows 20 banks apart keep a fragment's 32 words apart
template <bool GATED>
__global__ void __launch_bounds__(256) tile_kernel(const Linear l, int tn) {
  __shared__ __align__(16) uint16_t xs[128][kPitch], ws[128][kPitch];
  __shared__ int src[128];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
  const int wm = (warp & 3) * 32, wn = (warp >> 2) * 64;
  tc::pdl_trigger();
  tc::pdl_wait();
  Walk walk;
  walk.start(l, 7, 1, tn);
  Tile t;
  const uint16_t* x = reinterpret_cast<const uint16_t*>(l.x);
  for (long long i = blockIdx.x; i < 0x40000000 && walk.seek((int)i, t); i += gridDim.x) {
    const long long n0 = t.n * (GATED ? 64ll : 128ll);
    const uint16_t* w = reinterpret_cast<const uint16_t*>(l.w) + t.group * l.group_stride;
    __syncthreads();
    if (threadIdx.x < 128) src[threadIdx.x] = (int)threadIdx.x < t.rows ? source_row(l, t.row + threadIdx.x) : -1;
    __syncthreads();
    uint16_t xv[16], wv[16];
    auto load = [&](long long k) {  // this lane's k of rows warp, warp + 8, ..
#pragma unroll
      for (int u = 0; u < 16; ++u) {
        const int r = warp + 8 * u, from = src[r];
        // gated: rows 16 f .. 16 f + 7 of the tile are gate rows, the next eight their up rows
        const long long n = n0 + (GATED ? r / 16 * 8 + r % 8 : r);
        xv[u] = from >= 0 && k < l.k ? x[from * l.x_stride + k] : 0;
        wv[u] = n < l.n && k < l.k ? w[(n + (GATED && r & 8 ? l.n : 0)) * l.w_stride + k] : 0;
      }
    };
    float acc[2][8][4] = {};
    load(lane);
    for (long long k0 = 0; k0 < l.k; k0 += 32) {
#pragma unroll
      for (int u = 0; u < 16; ++u) {
        xs[warp + 8 * u][lane] = xv[u];
        ws[warp + 8 * u][lane] = wv[u];
      }
      __syncthreads();
      if (k0 + 32 < l.k) load(k0 + 32 + lane);
#pragma unroll
      for (int k = 0; k < 32; k += 16) {
        uint32_t a[2][4];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            a[m][q] = *reinterpret_cast<const uint32_t*>(&xs[wm + 16 * m + g + 8 * (q & 1)][k + 2 * t4 + 8 * (q >> 1)]);
#pragma unroll
        for (int n = 0; n < 8; ++n) {
          const uint32_t b0 = *reinterpret_cast<const uint32_t*>(&ws[wn + 8 * n + g][k + 2 * t4]);
          const uint32_t b1 = *reinterpret_cast<const uint32_t*>(&ws[wn + 8 * n + g][k + 2 * t4 + 8]);
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            float part[4] = {};
            mma_16x8(part, a[m][0], a[m][1], a[m][2], a[m][3], b0, b1);
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[m][n][q] += part[q];
          }
        }
      }
      __syncthreads();
    }
    with_act(l.act, [&](auto act) {
#pragma unroll
      for (int n = 0; n < 8; n += GATED ? 2 : 1)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const long long at = n0 + (GATED ? wn / 2 + 4 * n : wn + 8 * n) + 2 * t4 + e;
          if (at >= l.n) continue;
          float bias = 0.f, ubias = 0.f;
          if (l.bias) {
            const __nv_bfloat16* b = l.bias + (long long)t.group * l.n * (GATED ? 2 : 1) + at;
            bias = __bfloat162float(b[0]);
            if (GATED) ubias = __bfloat162float(b[l.n]);
          }
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int r = wm + 16 * m + g + 8 * h;
              if (src[r] < 0) continue;
              float y = act(acc[m][n][2 * h + e] + bias);
              if (GATED) y *= acc[m][n + (GATED ? 1 : 0)][2 * h + e] + ubias;
              finish(l, t.row + r, at, y);
            }
        }
    });
  }
}

__device__ __forceinline__ void dot8(float& acc, const uint4& w, const uint4& x) {
  const uint32_t a[4] = {w.x, w.y, w.z, w.w}, b[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    acc = fmaf(__uint_as_float(a[j] << 16), __uint_as_float(b[j] << 16), acc);
    acc = fmaf(__uint_as_float(a[j] & 0xffff0000u), __uint_as_float(b[j] & 0xffff0000u), acc);
  }
}
// Sums of N values over the lanes: lane l keeps that of value l * N / 32 (in its highest bits).  Half the values change
// hands at each of the first steps: N - 1 + log2(32 / N) shuffles for N * 5.
template <int N>
__device__ __forceinline__ float lane_sums(float (&v)[N]) {
  const int lane = threadIdx.x & 31;
  int o = 16;
#pragma unroll
  for (int m = N / 2; m >= 1; m >>= 1, o >>= 1) {
    const bool up = lane & o;
#pragma unroll
    for (int i = 0; i < m; ++i) {
      const float got = __shfl_xor_sync(kAll, up ? v[i] : v[i + m], o);
      v[i] = (up ? v[i + m] : v[i]) + got;
    }
  }
  for (; o > 0; o >>= 1) v[0] += __shfl_xor_sync(kAll, v[0], o);
  return v[0];
}

// R rows of x (grouped: the place blockIdx.y alone).  A CTA takes NB rows of
// weights per part of n (of each matrix half as many if gated); `kw` of its warps share a part, each a
// slice of K at a time, the slices of x in registers.
template <int R, bool GATED, int THREADS>
__global__ void __launch_bounds__(THREADS, kDotCtas<R, GATED, THREADS>) dot_kernel(const Linear l, int kw) {
  constexpr int kWarps = THREADS / 32, U = Dots<R>::U, NB = Dots<R>::NB, H = GATED ? NB / 2 : NB;  // H results a part
  __shared__ int found;
  __shared__ float sums[kWarps][NB * R];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  tc::pdl_trigger();
  if (threadIdx.x == 0) found = 0;
  tc::pdl_wait();
  int group = 0;
  long long row0 = 0;  // of out
  const __nv_bfloat16* x = l.x;
  if (l.offsets) {
    // the last group that starts at p or before: as many offsets as are not above p, counted by the block, all loads
    // in flight
    const int p = blockIdx.y, src = source_row(l, p);
    int below = 0;
    __syncthreads();
    for (int g0 = threadIdx.x; g0 <= l.groups; g0 += 4 * THREADS) {
      int at[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) at[u] = g0 + u * THREADS <= l.groups ? l.offsets[g0 + u * THREADS] : 0x7fffffff;
#pragma unroll
      for (int u = 0; u < 4; ++u) below += at[u] <= p;
    }
    below = __reduce_add_sync(kAll, below);
    if (lane == 0 && below) atomicAdd(&found, below);
    __syncthreads();
    group = found - 1;
    if (group < 0 || group >= l.groups || src < 0) return;
    x += src * l.x_stride;
    row0 = p;
  }
  const int part = warp / kw, slice = warp % kw, parts = kWarps / kw;
  const long long n0 = ((long long)blockIdx.x * parts + part) * H;
  // thread i of a part finishes result i % H of row i / H; what it needs is loaded now
  const int mine = slice * 32 + lane;
  const long long n = n0 + mine % H;
  const int row = mine / H;
  const bool ends = mine < H * R && n < l.n && (l.offsets || row < l.rows);
  float bias = 0.f, ubias = 0.f, res = 0.f;
  if (ends) {
    if (l.bias) {
      const __nv_bfloat16* b = l.bias + (long long)group * l.n * (GATED ? 2 : 1);
      bias = __bfloat162float(b[n]);
      if (GATED) ubias = __bfloat162float(b[l.n + n]);
    }
    if (l.res) res = load_res(l, (row0 + row) * l.res_stride + n);
  }
  const uint4 *w[NB], *xr[R];
  const __nv_bfloat16* base = l.w + group * l.group_stride;
#pragma unroll
  for (int j = 0; j < NB; ++j) {  // rows past the matrix are its last
    const long long at = n0 + j % H < l.n ? n0 + j % H : l.n - 1;
    w[j] = reinterpret_cast<const uint4*>(base + (at + (j >= H ? l.n : 0)) * l.w_stride) + lane;
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
    xr[r] = reinterpret_cast<const uint4*>(x + (l.offsets || r < l.rows ? r : l.rows - 1) * l.x_stride) + lane;
  float acc[NB * R] = {};
  const int pieces = l.k / 8;
  int i = slice * (32 * U);
  for (; i + 32 * U <= pieces; i += kw * 32 * U) {
    uint4 p[NB][U], v[R][U];
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int u = 0; u < U; ++u) p[j][u] = w[j][i + 32 * u];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int u = 0; u < U; ++u) v[r][u] = xr[r][i + 32 * u];
#pragma unroll
    for (int j = 0; j < NB; ++j)
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int u = 0; u < U; ++u) dot8(acc[j * R + r], p[j][u], v[r][u]);
  }
  for (int u = 0; u < U; ++u)  // the slice that is not whole
    if (i + 32 * u + lane < pieces)
#pragma unroll
      for (int j = 0; j < NB; ++j)
#pragma unroll
        for (int r = 0; r < R; ++r) dot8(acc[j * R + r], w[j][i + 32 * u], xr[r][i + 32 * u]);
  const float sum = lane_sums(acc);
  if (lane % (32 / (NB * R)) == 0) sums[warp][lane / (32 / (NB * R))] = sum;
  __syncthreads();
  if (!ends) return;
  float y = bias, up = ubias;
  for (int k = 0; k < kw; ++k) {
    y += sums[part * kw + k][(mine % H) * R + row];
    if (GATED) up += sums[part * kw + k][(H + mine % H) * R + row];
  }
  with_act(l.act, [&](auto act) {
    y = act(y);
    if (GATED) y *= up;
    store_out(l, (row0 + row) * l.out_stride + n, l.res ? fmaf(l.alpha, y, res) : l.alpha * y);
  });
}

template <int R, int THREADS>
cudaError_t launch_dots(const Linear& l, long long sms, cudaStream_t s) {
  constexpr int kWarps = THREADS / 32;
  // Slices of K as there are whole ones; where a CTA has its group to look up first, as long as all CTAs run at once (two
  // places of 2 x 512 x 2,048: 5.1 us in four slices, 6.5 in two; eight: 9.6 and 8.8).
  const int H = l.gated ? Dots<R>::NB / 2 : Dots<R>::NB;
  auto ctas = [&](int k) { return (l.n + (long long)(kWarps / k) * H - 1) / ((kWarps / k) * H) * l.rows; };
  const long long at_once = sms * (l.gated ? kDotCtas<R, true, THREADS> : kDotCtas<R, false, THREADS>);
  int kw = 1;
  while (kw < kWarps && l.k >= 2 * kw * 256 * Dots<R>::U && (!l.offsets || kw < 2 || ctas(2 * kw) <= at_once))
    kw *= 2;
  const long long per = (long long)(kWarps / kw) * H, blocks = (l.n + per - 1) / per;
  const dim3 grid((unsigned)blocks, l.offsets ? l.rows : 1), block(THREADS);
  if (l.gated) return tc::launch_early(dot_kernel<R, true, THREADS>, grid, block, 0, s, l, kw);
  return tc::launch_early(dot_kernel<R, false, THREADS>, grid, block, 0, s, l, kw);
}
// Four times the warps, and slices of K, where few results have long sums (1,024 x 8,192: 5.1 us for 8.2).
template <int R>
cudaError_t launch_dots(const Linear& l, long long sms, cudaStream_t s) {
  const bool thin = !l.offsets && l.k >= 4096 && l.n <= 2 * sms * (l.gated ? Dots<R>::NB / 2 : Dots<R>::NB);
  return thin ? launch_dots<R, 4 * kDotThreads>(l, sms, s) : launch_dots<R, kDotThreads>(l, sms, s);
}

// Up to 8 TN rows of x (the last again where there are fewer).  A CTA takes 16 rows of weights (8 gate rows and
// their up rows), its warps 32 of K in turn, from memory to registers in the order of the MMA's operands: which
// of K an operand's place holds is free as long as it is the same for both, so lane 4 g + t loads 16 bytes of row g,
// from t * 8 on, and these are its places of two MMAs.
template <int TN, bool GATED, int WARPS>
__global__ void __launch_bounds__(WARPS * 32) stream_kernel(const Linear l) {
  constexpr int U = 4, OUT = GATED ? 8 : 16;  // U: steps of K in flight
  constexpr int kValues = OUT * 8 * TN, kPer = (kValues + WARPS * 32 - 1) / (WARPS * 32);
  __shared__ float sums[WARPS][TN][16][9];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  tc::pdl_trigger();
  tc::pdl_wait();
  const long long n0 = (long long)blockIdx.x * OUT;
  const long long ra = n0 + g < l.n ? n0 + g : l.n - 1, rb = GATED ? ra + l.n : n0 + g + 8 < l.n ? n0 + g + 8 : l.n - 1;
  const uint4* wa = reinterpret_cast<const uint4*>(l.w + ra * l.w_stride) + t;
  const uint4* wb = reinterpret_cast<const uint4*>(l.w + rb * l.w_stride) + t;
  const uint4* xr[TN];
#pragma unroll
  for (int j = 0; j < TN; ++j) xr[j] = reinterpret_cast<const uint4*>(l.x + min(8 * j + g, l.rows - 1) * l.x_stride) + t;
  const int pieces = l.k / 8;  // of 16 bytes; a step is four
  float c[TN][4] = {};
  auto add = [&](const uint4& a, const uint4& b, const uint4 (&v)[TN]) {
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      mma_16x8(c[j], a.x, b.x, a.y, b.y, v[j].x, v[j].y);
      mma_16x8(c[j], a.z, b.z, a.w, b.w, v[j].z, v[j].w);
    }
  };
  constexpr int kStep = 4 * WARPS;
  int i = 4 * warp;
  for (; i + kStep * (U - 1) + 4 <= pieces; i += kStep * U) {
    uint4 a[U], b[U];
#pragma unroll
    for (int u = 0; u < U; ++u) a[u] = wa[i + kStep * u], b[u] = wb[i + kStep * u];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      uint4 v[TN];
#pragma unroll
      for (int j = 0; j < TN; ++j) v[j] = xr[j][i + kStep * u];
      add(a[u], b[u], v);
    }
  }
  for (; i < pieces; i += kStep) {
    uint4 a = make_uint4(0, 0, 0, 0), b = a, v[TN];
    const bool in = i + t < pieces;
    if (in) a = wa[i], b = wb[i];
#pragma unroll
    for (int j = 0; j < TN; ++j) {
      v[j] = make_uint4(0, 0, 0, 0);
      if (in) v[j] = xr[j][i];
    }
    add(a, b, v);
  }
#pragma unroll
  for (int j = 0; j < TN; ++j) {
    sums[warp][j][g][2 * t] = c[j][0];
    sums[warp][j][g][2 * t + 1] = c[j][1];
    sums[warp][j][g + 8][2 * t] = c[j][2];
    sums[warp][j][g + 8][2 * t + 1] = c[j][3];
  }
  __syncthreads();
  with_act(l.act, [&](auto act) {
#pragma unroll
    for (int z = 0; z < kPer; ++z) {
      const int i = threadIdx.x + z * WARPS * 32, r = i % OUT, token = i / OUT;
      const long long n = n0 + r;
      if (i >= kValues || token >= l.rows || n >= l.n) continue;
      float y = 0.f, up = 0.f;
#pragma unroll
      for (int k = 0; k < WARPS; ++k) {
        y += sums[k][token / 8][r][token % 8];
        if (GATED) up += sums[k][token / 8][r + 8][token % 8];
      }
      if (l.bias) {
        y += __bfloat162float(l.bias[n]);
        if (GATED) up += __bfloat162float(l.bias[l.n + n]);
      }
      y = act(y);
      if (GATED) y *= up;
      finish(l, token, n, y);
    }
  });
}

template <int TN>
cudaError_t launch_stream(const Linear& l, bool thin, cudaStream_t s) {
  const int per = l.gated ? 8 : 16;
  const dim3 grid((unsigned)((l.n + (long long)per - 1) / per));
  auto go = [&](auto kern, int warps) { return tc::launch_early(kern, grid, dim3(warps * 32), 0, s, l); };
  if (thin) return l.gated ? go(stream_kernel<TN, true, 32>, 32) : go(stream_kernel<TN, false, 32>, 32);
  return l.gated ? go(stream_kernel<TN, true, 16>, 16) : go(stream_kernel<TN, false, 16>, 16);
}

// A few rows of any layout: a warp per result's weights, an element a lane, four rows of x at a time.
template <bool GATED>
__global__ void __launch_bounds__(256) any_kernel(const Linear l) {
  const int lane = threadIdx.x & 31;
  const long long n = (long long)blockIdx.x * 8 + (threadIdx.x >> 5);
  tc::pdl_trigger();
  tc::pdl_wait();
  if (n >= l.n) return;
  const __nv_bfloat16 *w = l.w + n * l.w_stride, *up = w + (long long)l.n * l.w_stride;
  for (int r0 = 0; r0 < l.rows; r0 += 4) {
    float a[4] = {}, b[4] = {};
    const __nv_bfloat16* x[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) x[r] = l.x + min(r0 + r, l.rows - 1) * l.x_stride;
#pragma unroll 8
    for (int k = lane; k < l.k; k += 32) {
      const float wv = __bfloat162float(w[k]), uv = GATED ? __bfloat162float(up[k]) : 0.f;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float xv = __bfloat162float(x[r][k]);
        a[r] = fmaf(wv, xv, a[r]);
        if (GATED) b[r] = fmaf(uv, xv, b[r]);
      }
    }
    const float sum = lane_sums(a), usum = GATED ? lane_sums(b) : 0.f;  // row lane / 8's
    if (lane % 8 == 0 && r0 + lane / 8 < l.rows)
      with_act(l.act, [&](auto act) {
        float y = act(sum + (l.bias ? __bfloat162float(l.bias[n]) : 0.f));
        if (GATED) y *= usum + (l.bias ? __bfloat162float(l.bias[l.n + n]) : 0.f);
        finish(l, r0 + lane / 8, n, y);
      });
  }
}

template <bool GATED>
cudaError_t launch_tiles(const Linear& l, int sms, cudaStream_t s) {
  const int per = GATED ? 64 : 128, tn = (int)((l.n + (long long)per - 1) / per);
  const long long most = most_tiles(l, 7, tn);
  if (most > 0x3fffffff) return cudaErrorInvalidValue;
  const long long grid = most < 8ll * sms ? most : 8ll * sms;
  return tc::launch_early(tile_kernel<GATED>, dim3((unsigned)grid), dim3(256), 0, s, l, tn);
}

}  // namespace

cudaError_t launch_linear(const Linear& call, cudaStream_t s) {
  Linear l = call;
  division_of(l.per_row, l.per_mul, l.per_shift);
  tc::DeviceInfo d;
  const cudaError_t e = tc::device_info(&d);
  if (e != cudaSuccess) return e;
  const bool whole = l.k % 8 == 0 && l.x_stride % 8 == 0 && l.w_stride % 8 == 0 && l.group_stride % 8 == 0 &&
                     ((reinterpret_cast<uintptr_t>(l.x) | reinterpret_cast<uintptr_t>(l.w)) & 15) == 0;
  // Places one by one while they are few, or most have a group to themselves (24 / 48 places over 256 experts of
  // 2 x 512 x 2,048: 19.6 / 34.2 us, in tiles 23.8 / 35.8; 48 over 64 of 2 x 1,024 x 4,096: 96 and 87).  Each place reads
  // its whole matrix: more places than groups read some again, from L2 or not, and no more than 64 MiB of it (over one group,
  // dot products / tiles: 16 places of 2 x 512 x 2,048 9.2 / 9.6 us, of 4,096 x 1,024 20.1 / 7.3; 4 and 16 of 2 x 1,024 x 4,096
  // 8.5 / 15.0 and 21.9 / 15.1; 2 and 16 of 4,096 x 8,192 15.5 / 24.6 and 69.2 / 24.6, of 16,384 x 8,192 80 / 45 and 581 / 46;
  // over 16 groups of 2 x 1,024 x 4,096: 8 places 24.0 / 24.1, 16 45.3 / 42.9).
  const long long read = (long long)l.n * (l.gated ? 2 : 1) * l.k * 2;  // by a place
  const bool few = l.rows <= 16 ? l.rows <= l.groups || read <= (1ll << 26) / (l.rows - 1)
                                : l.rows <= 48 && 4 * l.rows <= l.groups;
  if (whole && l.offsets && few) return launch_dots<1>(l, d.sms, s);
  if (whole && !l.offsets && l.rows <= kDotRows)
    return l.rows == 1 ? launch_dots<1>(l, d.sms, s) : launch_dots<2>(l, d.sms, s);
  // The streaming kernel where its CTAs, one per 16 rows of weights, are at most two an SM and K gives each no more than
  // a few rounds (4,096 x 4,096: 9.2 us for 4 rows, 9.9 for 16, and 11.2 and 12.2 in the tiles below; 8 x 2 x 512 x 2,048
  // gated: 4.2 and 6.5), twice the warps where they are at most one and K is long (8 x 1,024 x 8,192: 8.1 us, in the tiles
  // 11); else the tiles (16 x 16,384 x 2,048: 14.1 us, here 19.3).
  const long long blocks = (l.n + (l.gated ? 7ll : 15ll)) / (l.gated ? 8 : 16);
  const bool thin = blocks <= d.sms && l.k >= 4096;
  if (whole && !l.offsets && l.rows <= kStreamRows && (thin ? l.k <= 8192 : blocks <= 2ll * d.sms && l.k <= 4096))
    return l.rows <= 8 ? launch_stream<1>(l, thin, s) : launch_stream<2>(l, thin, s);
  // What the tensor-core kernel's copies address: strides below 2^40 bytes, gathered rows in 32 bits of 16-byte
  // pieces; and a tile's K within what its waits allow (512 cycles for 64 of K).
  const long long most = 1ll << 38;
  const bool near = l.x_stride < most && l.w_stride < most / (l.gated ? l.n : 1) && l.group_stride < most &&
                    (!l.order || l.x_rows <= (1ll << 35) / l.x_stride) && l.k <= 1 << 26;
  if (whole && near && (!l.gated || l.n % 16 == 0)) return launch_linear_tc(l, d.sms, s);
  if (!l.offsets && l.rows <= kStreamRows && l.k <= 1 << 30) {
    const dim3 grid((unsigned)((l.n + 7ll) / 8)), block(256);
    if (l.gated) return tc::launch_early(any_kernel<true>, grid, block, 0, s, l);
    return tc::launch_early(any_kernel<false>, grid, block, 0, s, l);
  }
  return l.gated ? launch_tiles<true>(l, d.sms, s) : launch_tiles<false>(l, d.sms, s);
}

}  // namespace moe

// linear_tc.cu -- the bf16 products on the tensor cores: out = epilogue(x w^T), dense or
// one product per group, for operands in rows of whole 16-byte pieces.
//
// The weights are the MMA's 128 rows (256 with a CTA pair, CG = 2), the tokens its
// columns: a tile takes as many tokens as are there, up to NT and a multiple of 16, so that a
// ragged group costs what its rows cost, and one tile shape serves groups of any size.
// A stage of the pipeline is 128 bytes of every row (64 of K, four MMAs).  CTAs (or pairs)
// are persistent and take tiles in turn; the groups' offsets are read on the device.  Warps:
//   0..7  epilogue: tensor memory -> shared memory -> bias, activation, gate, residual -> out.
//         Warp w takes lanes 32 (w % 4) .. (its results' n), blocks w / 4, w / 4 + 2, .. of the
//         tokens.  Two accumulators alternate, so the next tile's MMAs run beside it;
//   8     TMA loads of the weights (tokens: boxes of 32 rows, or of all);
//   9     MMAs (the first CTA's of a pair);
//   10,11 tokens by the order's indices, where there is one; else their boxes, and half of a gated
//         tile's weights.
// Gated products: a CTA's 128 rows are 64 gate rows and their 64 up rows in runs of 16
// (boxes of 16 gate and 16 up rows), so that the two halves of a result are one warp's.
// What bounds it: 8,192 x 8,192 x 4,096 with bias, tanh GELU and residual 305 us, the tensor pipe busy 92% of
// the cycles (plain 281 us, 1,957 TFLOP/s); experts' gate and up (256 of 2 x 512 x 2,048, 65,536 gathered
// rows) 255 to 275 us, 11.4 TB/s from L2 to the SMs; down products (4,096 x 1,024) HBM, 96%.
// Sums: the tensor cores add with truncation, an error that grows with the chain of additions;
// the sum is taken in as many parts of K, up to four, as leave room for two accumulators.  Where these are too long
// (kPart) the parts go through three accumulators in turn, and the epilogue's warps add each to a sum of their own.
// Where tiles are few, `split` CTAs (pairs) of a cluster share a tile: each sums its part of K,
// then its share of the rows over the parts in ascending order.
// Every wait is bounded; on a timeout the CTA reports it, drains its copies and MMAs, frees
// its tensor memory and returns.  A tile is stored whole and right or not at all.
#include "linear.cuh"
#include "tc.cuh"

namespace moe {
namespace {

using namespace tc;
using namespace lin;

constexpr int kEpiWarps = 8, kTmaWarp = 8, kMmaWarp = 9, kRowWarp = 10, kThreads = 384;
constexpr long long kLandCycles = 2000 * 1000;
// K of one chain at most, for results of fp32 and of bf16.  Chains of 256 are off by 2.4e-7 of the norm of the sums, whatever
// the whole K, one of 4,096 by 4.4e-6 (a plain fp32 form at K 1,024 / 4,096 / 16,384: 2.5e-7 / 6.1e-7 / 1.5e-6); the rounding to
// bf16 is off by 1.7e-3.  Chains of 256 / 512 / one in tiles of 256 tokens: 65,536 rows of 256 groups, N 1,024, at K 1,024
// 188 / 175 / 150 us, at 2,048 318 / 300 / 254; 8,192 x 8,192 at K 4,096 350 / 338 / 294, at 512 97 / 76.
constexpr int kPart = 256, kPartBf16 = 65536;
constexpr int kMaxCluster = 4;  // CTAs; eights do not all find room at once

template <int NT, int CG>
struct Shape {
  static constexpr int kX = NT / CG;                     // token rows a CTA loads
  // 64-element slabs of K in a stage: two where a stage's MMAs would not outlast its issue
  static constexpr int kSub = NT == 256 ? 1 : 2;
  static constexpr int kSlab = 128 * 128 + kX * 128;
  static constexpr int kStage = kSub * kSlab;
  static constexpr int W = NT == 32 ? 16 : 32;           // tokens the epilogue takes at a time
  static constexpr int kTurn = kEpiWarps * W * 128;      // their sums
  static constexpr int kFit = (226 * 1024 - 2048 - kTurn) / kStage;
  static constexpr int kStages = kFit > 12 ? 12 : kFit;
  static constexpr int kChains = 256 / NT < 4 ? 256 / NT : 4;
  static constexpr int kCols = 2 * kChains * NT;         // of tensor memory
  static constexpr int kSmem = kStages * kStage + kTurn + 1024;
  static constexpr int kPitch = NT + 4;                  // of a split's sums
  static_assert(kCols <= 512 && (kCols & (kCols - 1)) == 0 && kStage % 1024 == 0, "tile shape");
  static_assert(NT == 256 || kCols >= 4 * NT, "room for a long sum");
  static_assert(kStages * kStage + kTurn >= 128 * kPitch * 4 * (CG == 1 ? 7 : 6) / 4, "room for a split's sums");
};

struct Args {
  Linear l;
  int tn;     // tiles of n
  int tiles, width;  // of tokens, in a dense product
  int shift;  // a group's tiles have up to 1 << shift tokens
  int nk;     // stages of K
  int split;  // parts of K
  int part;   // stages of K of a chain at most
  int wide;   // four neighbouring results of out and res are one aligned access
};

template <int ST>
struct Ctl {
  uint64_t full[ST], empty[ST], landed[ST];  // landed: gathered rows of x
  uint64_t acc_full[3], acc_empty[3], drain, sums;
  uint32_t tmem;
  int abort_flag, epi_ok[2];  // epi_ok: the epilogue's waits in turn
};

#define MOE_LIN_LOAD(cg, dim, coords)                                                             \
  asm volatile("cp.async.bulk.tensor." dim cg ".mbarrier::complete_tx::bytes [%0], [%1, {" coords \
               "}], [%2];"
// rows n .. n + 127 of a group's weights
template <int CG>
__device__ __forceinline__ void load_rows(void* dst, const CUtensorMap* map, int x, int n, int g, uint32_t bar) {
  if constexpr (CG == 1)
    MOE_LIN_LOAD(".shared::cluster.global", "3d", "%3, %4, %5")
    ::"r"(sa(dst)), "l"(map), "r"(bar), "r"(x), "r"(n), "r"(g) : "memory");
  else
    MOE_LIN_LOAD(".cta_group::2.shared::cluster.global", "3d", "%3, %4, %5")
    ::"r"(sa(dst)), "l"(map), "r"(bar), "r"(x), "r"(n), "r"(g) : "memory");
}
// 16 gate rows and their 16 up rows; c: n / 16
template <int CG>
__device__ __forceinline__ void load_gated(void* dst, const CUtensorMap* map, int x, int c, int g, uint32_t bar) {
  if constexpr (CG == 1)
    MOE_LIN_LOAD(".shared::cluster.global", "5d", "%3, %4, %5, %6, %7")
    ::"r"(sa(dst)), "l"(map), "r"(bar), "r"(x), "r"(0), "r"(c), "r"(0), "r"(g) : "memory");
  else
    MOE_LIN_LOAD(".cta_group::2.shared::cluster.global", "5d", "%3, %4, %5, %6, %7")
    ::"r"(sa(dst)), "l"(map), "r"(bar), "r"(x), "r"(0), "r"(c), "r"(0), "r"(g) : "memory");
}
#undef MOE_LIN_LOAD

// 16 bytes (or zeros) to shared memory; an arrival once all such copies of this thread have landed
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copies_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(sa(bar)) : "memory");
}
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }
__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

template <int CG>
__device__ __forceinline__ void mma(uint32_t d, uint64_t w, uint64_t x, uint32_t id, uint32_t acc) {
  if constexpr (CG == 1)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(w), "l"(x), "r"(id), "r"(acc)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
        " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
        "l"(w), "l"(x), "r"(id), "r"(acc)
        : "memory");
}
// bf16 operands, both K-major, fp32 sums, m x n
__device__ __forceinline__ uint32_t idesc(int m, int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}

// W tokens of the warp's lanes, the sums of n chains added up in order: the first at `at`, the others `step` on each
template <int W>
__device__ __forceinline__ void read_sums(uint32_t at, uint32_t step, int n, uint32_t (&v)[W]) {
  uint32_t u[W];
  tmem_ld(at, v);
  if (n > 1) tmem_ld(at + step, u);
  tmem_wait_ld();
  for (int k = 1; k < n; ++k) {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) + __uint_as_float(u[i]));
    if (k + 1 < n) {
      tmem_ld(at + (k + 1) * step, u);
      tmem_wait_ld();
    }
  }
}

// The accumulators in turn, as the MMAs fill them and the epilogue takes them.
template <int N>
struct Turn {
  int b = 0, par = 0;  // par: of this round
  __device__ __forceinline__ void next() {
    b = b + 1 == N ? 0 : b + 1;
    par ^= b == 0;
  }
};

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void sts(uint32_t saddr, uint32_t v) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(saddr), "r"(v) : "memory");
}

__device__ __forceinline__ float lds(uint32_t saddr) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(saddr));
  return v;
}

// The epilogue of a warp: blocks of W tokens, its 32 lanes' sums turned in shared memory so that
// a lane finishes four neighbouring results of a token (1 store of 8 or 16 bytes, and as
// large a load of the residual, for four scattered ones).  Rows of 32 floats; odd tokens
// have their halves exchanged, which keeps the reads of 16 gate or up sums off each other's banks.
// A lane's tokens of a block are `step` apart, an even number, so its places are fixed.  Blocks of 32 have half
// the chain of latencies of 16 (8,192 x 8,192 x 512: 84 us, so 72).
template <int W>
struct Epilogue {
  const Linear& l;
  const bool gated, f32;
  const int lane, token, step;  // first of the lane's tokens in a block
  const uint32_t put0, put1;    // shared memory: this lane's sums of even and odd tokens
  const uint32_t get_a;         // the four sums of its first token; their up sums are 64 bytes on or back
  const long long out_step, res_step, es;  // bytes between the lane's rows, of an element
  // Where the lanes' results are all below n and aligned: four of a token each.  Else one of each token (of
  // every second one if gated), neighbours in neighbouring lanes.
  bool wide, in;                // in: a narrow lane's result is below n
  char* out;                    // the lane's first result of the tile
  const char* res;
  float bias[4], ubias[4];

  __device__ __forceinline__ Epilogue(const Linear& l_, uint32_t buf, int lane_)
      : l(l_), gated(l_.gated), f32(l_.f32), lane(lane_), token(l_.gated ? lane_ >> 2 : lane_ >> 3),
        step(l_.gated ? 8 : 4), put0(buf + 4 * lane_), put1(buf + 128 + 4 * (lane_ ^ 16)),
        get_a(buf + token * 128 + 16 * ((l_.gated ? lane_ & 3 : lane_ & 7) ^ (token & 1 ? 4 : 0))),
        out_step(step * l_.out_stride * (l_.f32 ? 4 : 2)),
        res_step(step * l_.res_stride * (l_.f32 ? 4 : 2)), es(l_.f32 ? 4 : 2) {}

  // n0: first result of the warp's lanes; row: the tile's first
  __device__ __forceinline__ void start(long long n0, long long row, int group, bool aligned) {
    wide = aligned && n0 + (gated ? 16 : 32) <= l.n;
    const long long n = n0 + (wide ? 4 * (gated ? lane & 3 : lane & 7) : gated ? lane & 15 : lane);
    in = n < l.n;
    row += wide ? token : gated ? lane >> 4 : 0;
    out = static_cast<char*>(l.out) + (row * l.out_stride + n) * es;
    res = static_cast<const char*>(l.res) + (l.res ? (row * l.res_stride + n) * es : 0);
    const __nv_bfloat16* b = l.bias ? l.bias + (long long)group * l.n * (gated ? 2 : 1) + n : nullptr;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bool here = b && in && (wide || j == 0);
      bias[j] = here ? __bfloat162float(b[j]) : 0.f;
      ubias[j] = here && gated ? __bfloat162float(b[l.n + j]) : 0.f;
    }
  }
  // The residual of the warp's blocks from token n0 on into L2, while the sums are made (2,048 x 2,048 x 2,048: 23.9 us,
  // so 21.7).
  __device__ __forceinline__ void prefetch(int n0, int rows) const {
    if (!wide) return;
    for (; n0 < rows; n0 += 2 * W)
      for (int t = token; t < W; t += step)
        if (n0 + t < rows)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(res + (n0 + t - token) * l.res_stride * es));
  }
  // The residual of the lane's results of the block at token n0, in the bits it is loaded in until it is used:
  // nothing waits for it before.
  __device__ __forceinline__ void fetch(int n0, uint32_t mask, uint32_t (&r)[W / 4][4]) const {
    const char* p = res + n0 * l.res_stride * es;
    if (wide) {
#pragma unroll
      for (int k = 0; k < W / 4; ++k)
        if ((k < W / 8 || !gated) && (mask >> (token + k * step) & 1)) {
          const char* q = p + k * res_step;
          if (f32) {
            const uint4 u = *reinterpret_cast<const uint4*>(q);
            r[k][0] = u.x, r[k][1] = u.y, r[k][2] = u.z, r[k][3] = u.w;
          } else {
            const uint2 u = *reinterpret_cast<const uint2*>(q);
            r[k][0] = u.x, r[k][1] = u.y;
          }
        }
    } else {
      const int first = gated ? lane >> 4 : 0, by = gated ? 2 : 1;
#pragma unroll
      for (int i = 0; i < W; ++i)
        if (i * by < W && in && (mask >> (first + i * by) & 1)) {
          const char* q = p + i * by * l.res_stride * es;
          r[i / 4][i % 4] = f32 ? *reinterpret_cast<const uint32_t*>(q) : *reinterpret_cast<const uint16_t*>(q);
        }
    }
  }
  __device__ __forceinline__ void turn(const uint32_t (&v)[W]) const {
#pragma unroll
    for (int i = 0; i < W; i += 2) {
      sts(put0 + i * 128, v[i]);
      sts(put1 + i * 128, v[i + 1]);
    }
  }
  // A block, 16 tokens at a time.
  template <bool GATED, typename A>
  __device__ __forceinline__ void finish(A act, int n0, uint32_t mask, uint32_t (&r)[W / 4][4]) const {
    char* p = out + n0 * l.out_stride * es;
#pragma unroll 1
    for (int half = 0; half < W / 16; ++half) {
      if (wide) finish_wide<GATED>(act, p, half * 2048, mask, r);
      else finish_narrow<GATED>(act, p, half * 2048, mask, r);
      p += 16 * l.out_stride * es;
      mask >>= 16;
      if (W > 16 && l.res) {
#pragma unroll
        for (int k = 0; k < W / 8; ++k)
#pragma unroll
          for (int j = 0; j < 4; ++j) r[k][j] = GATED && k >= W / 16 ? 0 : r[k + (GATED ? W / 16 : W / 8)][j];
      }
    }
  }
  template <bool GATED, typename A>
  __device__ __forceinline__ void finish_wide(A act, char* p, int at, uint32_t mask,
                                              const uint32_t (&r)[W / 4][4]) const {
    constexpr int M = GATED ? 2 : 4;
    float y[M][4];
#pragma unroll
    for (int k = 0; k < M; ++k) {
      const float4 g = lds4(get_a + at + k * (GATED ? 1024 : 512));
      y[k][0] = g.x, y[k][1] = g.y, y[k][2] = g.z, y[k][3] = g.w;
    }
#pragma unroll
    for (int k = 0; k < M; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) y[k][j] = act(y[k][j] + bias[j]);
    if constexpr (GATED) {
#pragma unroll
      for (int k = 0; k < M; ++k) {
        const float4 u = lds4((get_a + at + k * 1024) ^ 64);
        y[k][0] *= u.x + ubias[0], y[k][1] *= u.y + ubias[1], y[k][2] *= u.z + ubias[2], y[k][3] *= u.w + ubias[3];
      }
    }
#pragma unroll
    for (int k = 0; k < M; ++k) {
#pragma unroll
      for (int j = 0; j < 4; ++j) y[k][j] *= l.alpha;
      if (l.res) {
        if (f32) {
#pragma unroll
          for (int j = 0; j < 4; ++j) y[k][j] += __uint_as_float(r[k][j]);
        } else {
          y[k][0] += __uint_as_float(r[k][0] << 16), y[k][1] += __uint_as_float(r[k][0] & 0xffff0000u);
          y[k][2] += __uint_as_float(r[k][1] << 16), y[k][3] += __uint_as_float(r[k][1] & 0xffff0000u);
        }
      }
      char* q = p + k * out_step;
      if (mask >> (token + k * step) & 1) {
        if (f32) *reinterpret_cast<float4*>(q) = make_float4(y[k][0], y[k][1], y[k][2], y[k][3]);
        else *reinterpret_cast<uint2*>(q) = make_uint2(pack2(y[k][0], y[k][1]), pack2(y[k][2], y[k][3]));
      }
    }
  }
  template <bool GATED, typename A>
  __device__ __forceinline__ void finish_narrow(A act, char* p, int half, uint32_t mask,
                                                const uint32_t (&r)[W / 4][4]) const {
    constexpr int BY = GATED ? 2 : 1;
    const int first = GATED ? lane >> 4 : 0;
    const long long by = BY * l.out_stride * es;
    uint32_t bit = 1u << first;
    // sums of token first + BY * i; gated, the up lanes' tokens are odd and turned
    uint32_t at = half + (GATED ? put0 - 4 * lane + first * 128 + 4 * ((lane & 15) ^ (first ? 16 : 0)) : put0);
    const uint32_t odd = GATED ? 0 : (4 * lane ^ 64) - 4 * lane;  // of an odd token's place, not gated
#pragma unroll
    for (int k = 0; k < 4 / BY; ++k, at += 512 * BY) {
#pragma unroll
      for (int j = 0; j < 4; ++j, p += by, bit <<= BY) {
        const uint32_t here = at + j * 128 * BY + (j & 1 ? odd : 0);
        float y = act(lds(here) + bias[0]);
        if (GATED) y *= lds(here ^ 64) + ubias[0];
        y *= l.alpha;
        if (l.res) y += __uint_as_float(f32 ? r[k][j] : r[k][j] << 16);
        if (in && (mask & bit)) {
          if (f32) *reinterpret_cast<float*>(p) = y;
          else *reinterpret_cast<__nv_bfloat16*>(p) = __float2bfloat16_rn(y);
        }
      }
    }
  }
};

// LONG: sums of more chains than an accumulator has.  Three accumulators of one chain each then, and the sum of the
// chains so far as a fourth, which the epilogue alone uses; else two of up to kChains.  (By a branch in one
// kernel: 8,192 x 8,192 x 1,024 fp32 in two chains 113 us, so 108.)
template <int NT, int CG, bool LONG>
__global__ void __launch_bounds__(kThreads, 1)
linear_kernel(const __grid_constant__ CUtensorMap wmap, const __grid_constant__ CUtensorMap xmap,
              const __grid_constant__ CUtensorMap xmap_all, const __grid_constant__ Args a) {
  using S = Shape<NT, CG>;
  constexpr int ST = S::kStages, W = S::W;
  extern __shared__ uint8_t raw[];
  uint8_t* stg = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  __shared__ Ctl<ST> c;
  const Linear& l = a.l;
  // the warp's number from a shuffle: known to be the same for all lanes, with what follows from it
  const int warp = __shfl_sync(kAll, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  // cluster: `split` parts of K, each CG CTAs; a lone CTA's cluster is itself
  const int crank = CG == 1 && a.split == 1 ? 0 : (int)cluster_rank();
  const int pair = crank % CG, first = crank - pair, part = crank / CG;
  const int team = CG * a.split;
  const int k_lo = (int)((long long)a.nk * part / a.split), k_hi = (int)((long long)a.nk * (part + 1) / a.split);
  const int n_k = k_hi - k_lo;
  constexpr int kAccs = LONG ? 3 : 2, kAcc = LONG ? NT : S::kChains * NT;  // accumulators, columns of one
  const int n_chains = S::kChains == 1 ? 1 : min(S::kChains, n_k), n_parts = LONG ? (n_k + a.part - 1) / a.part : 1;
  const int tile0 = blockIdx.x / team, step = gridDim.x / team;
  const uint16_t both = (uint16_t)(((1 << CG) - 1) << first);
  const bool gather = CG == 2 && l.order;  // groups take pairs

  pdl_trigger();
  if (threadIdx.x < ST) {
    const int i = threadIdx.x;
    mbar_init(&c.full[i], gather ? CG : 1);  // with the second CTA's gathered rows handed on
    mbar_init(&c.empty[i], 1);
    mbar_init(&c.landed[i], 64);
    if (i < 3) {
      mbar_init(&c.acc_full[i], 1);
      mbar_init(&c.acc_empty[i], kEpiWarps * CG);
    }
    if (i == 0) {
      mbar_init(&c.drain, 1);
      mbar_init(&c.sums, 1);
      c.abort_flag = 0;
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kTmaWarp && elect_one()) {  // the maps are on their way when the first copy reads them
    prefetch_map(&wmap);
    prefetch_map(gather ? &wmap : &xmap_all);
  }
  if (warp == kMmaWarp) tmem_alloc<CG>(&c.tmem, S::kCols);
  fence_before();
  __syncthreads();
  if (CG > 1) cluster_sync();  // the peer's barriers exist before anything arrives there
  else if (a.split > 1) cluster_arrive();  // waited for before anything goes to a peer
  fence_after();
  const uint32_t tmem = c.tmem;

  // the part of a tile's tokens that a CTA loads, a multiple of 8
  auto half = [](int rows) { return (rows + 15) / 16 * 16 / CG; };
  // a warp's tile and its next one, looked for while the first is under way
  Walk walk;
  Tile t, next;
  bool more = false, more_next = false;
  if (l.offsets) pdl_wait();
  if (warp >= kEpiWarps || a.split == 1) {  // a split's sums are exchanged below
    walk.start(l, a.shift, 16, a.tn, a.tiles, a.width);
    more = walk.seek(tile0, t);
  }
  if (!l.offsets) pdl_wait();

  if (warp == kTmaWarp || (warp >= kRowWarp && !gather && (warp == kRowWarp || l.gated))) {
    // Two or three warps, since an instruction takes one about 100 cycles: the weights' copies, the tokens', and half of
    // a gated tile's weights.
    const int j_lo = warp == kTmaWarp ? 0 : 2, j_hi = warp == kTmaWarp && !gather ? 2 : 4;
    int it = 0, s = 0;
    bool ok = true;
    for (int i = tile0; ok && more; t = next, more = more_next) {
      // boxes of 32 rows, or all the CTA has room for at once
      const int hx = half(t.rows);
      const bool all = hx > S::kX - 32;
      const int boxes = gather ? 0 : all ? S::kX / 32 : (hx + 31) / 32;
      const int bytes = CG * S::kSub * (128 * 128 + boxes * 4096);
      const int x0 = t.row + pair * hx, nt = t.n * CG + pair;
      for (int ks = k_lo; ks < k_hi; ++ks, ++it) {
        if (it >= ST && !warp_wait(&c.empty[s], (it / ST - 1) & 1, &c.abort_flag, a.l.status)) {
          ok = false;
          break;
        }
        const uint32_t bar = CG == 1 ? sa(&c.full[s]) : peer_addr(sa(&c.full[s]), first);
        if (elect_one()) {
          // a pair's copies all count on the first CTA's barrier
          if (warp == kTmaWarp && pair == 0) mbar_expect(&c.full[s], bytes);
#pragma unroll
          for (int q = 0; q < S::kSub; ++q) {
            uint8_t* p = stg + (size_t)s * S::kStage + q * S::kSlab;
            const int x = (ks * S::kSub + q) * 64;
            if (warp != kRowWarp) {
              if (l.gated) {
                for (int j = j_lo; j < j_hi; ++j) load_gated<CG>(p + j * 4096, &wmap, x, nt * 4 + j, t.group, bar);
              } else {
                load_rows<CG>(p, &wmap, x, nt * 128, t.group, bar);
              }
            } else if (all) {
              tma_load<CG>(p + 128 * 128, &xmap_all, x, x0, bar);
            } else {
              for (int j = 0; j < boxes; ++j) tma_load<CG>(p + 128 * 128 + j * 4096, &xmap, x, x0 + 32 * j, bar);
            }
          }
        }
        __syncwarp();
        s = s + 1 == ST ? 0 : s + 1;
        if (ks == k_lo) more_next = walk.seek(i += step, next);
      }
    }
    // The copies in flight land before the CTA ends, whichever warp may have given up.  A stage that others did not
    // get to is never full: this wait is a thousand times what a copy takes.
    if (pair == 0) {
      const long long t0 = clock64();
      for (int i = it > ST ? it - ST : 0; i < it; ++i)
        while (!mbar_test(&c.full[i % ST], (i / ST) & 1) && clock64() - t0 < kLandCycles) {
        }
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    if (pair == 0) {
      int s = 0;
      uint32_t full_par = 0;
      bool ok = true;
      const uint64_t w_base = desc_tile(sa(stg)), x_base = desc_tile(sa(stg) + 128 * 128);
      Turn<kAccs> acc;
      // an accumulator of the first round is free: the phase before a barrier's first one counts as over
      auto take = [&] { return warp_wait(&c.acc_empty[acc.b], acc.par ^ 1, &c.abort_flag, a.l.status); };
      for (int i = tile0; ok && more; t = next, more = more_next) {
        if (!take()) break;
        const uint32_t id = idesc(128 * CG, half(t.rows) * CG);
        uint32_t d = tmem + acc.b * kAcc;
        // the part of K being summed, its first stage, the next's
        int chain = 0, first_of = 0, next_of = LONG ? a.part : n_k / n_chains;
        for (int k = 0; k < n_k; ++k) {
          if ((LONG || S::kChains > 1) && k == next_of) {
            first_of = k;
            if constexpr (LONG) {
              if (elect_one()) mma_commit<CG>(&c.acc_full[acc.b], both);
              __syncwarp();
              acc.next();
              if (!take()) {
                ok = false;
                break;
              }
              next_of += a.part;
              d = tmem + acc.b * kAcc;
            } else {
              ++chain;
              next_of = n_k * (chain + 1) / n_chains;
              d += NT;
            }
          }
          if ((gather && !warp_wait(&c.landed[s], full_par, &c.abort_flag, a.l.status)) ||
              !warp_wait(&c.full[s], full_par, &c.abort_flag, a.l.status)) {
            ok = false;
            break;
          }
          if (gather) {
            fence_async_smem();
            __syncwarp();
          }
          fence_after();
          if (elect_one()) {
            const uint64_t w0 = w_base + (uint64_t)(s * (S::kStage / 16)), x0 = x_base + (uint64_t)(s * (S::kStage / 16));
#pragma unroll
            for (int j = 0; j < 4 * S::kSub; ++j) {  // 32 bytes of every row each
              const int at = j / 4 * (S::kSlab / 16) + j % 4 * 2;
              mma<CG>(d, w0 + at, x0 + at, id, j > 0 || k > first_of);
            }
            mma_commit<CG>(&c.empty[s], both);
          }
          __syncwarp();
          if (++s == ST) s = 0, full_par ^= 1;
          if (k == 0) more_next = walk.seek(i += step, next);
        }
        if (!ok) break;
        if (elect_one()) mma_commit<CG>(&c.acc_full[acc.b], both);
        __syncwarp();
        acc.next();
      }
      if (elect_one()) mma_commit<CG>(&c.drain, both);
      __syncwarp();
    } else if (gather) {
      // The second CTA's gathered rows, fenced and handed on to the first.  The arrival is the default one:
      // with .release.cluster it took 2,000 cycles beside copies in flight, four times a stage
      // (65,536 x 1,024 x 2,048 in 256 groups: 564 us, so 284); the rows are in this CTA's shared memory, in order
      // for its MMAs by the fence.
      int s = 0;
      uint32_t par = 0;
      bool ok = true;
      for (int i = tile0; ok && more; more = walk.seek(i += step, t))
        for (int k = 0; ok && k < n_k; ++k) {
          ok = warp_wait(&c.landed[s], par, &c.abort_flag, a.l.status);
          fence_async_smem();
          __syncwarp();
          if (ok && lane == 0) mbar_arrive_at(peer_addr(sa(&c.full[s]), first));
          if (++s == ST) s = 0, par ^= 1;
        }
      __syncwarp();
    }
    drain_bar(&c.drain, 0);  // every MMA has finished before the tensor memory is freed
    __syncwarp();
  } else if (warp >= kRowWarp) {
    // Rows of x by the order's indices: 16 bytes a lane, four rows a warp and instruction, in the
    // copies' swizzle.  A thread's copies arrive at `landed` by themselves; the warp that waits
    // there fences them for the MMAs.  (TMA's four-row gathers took about 70 cycles each, 2,200 a
    // stage of 128 rows; a fence by the copying threads waits for all their copies in flight.)
    if (gather) {
      constexpr int kPer = S::kX / 8;  // rows of a lane
      const int gw = warp - kRowWarp, chunk = lane & 7, r0 = 4 * gw + (lane >> 3);
      int it = 0, s = 0;
      bool ok = true;
      int order[kPer];  // of the tile's rows, loaded while the one before is copied
      auto look_up = [&](const Tile& z) {
#pragma unroll
        for (int j = 0; j < kPer; ++j)
          // past the tile its last row again (one row for all tiles would be one L2 slice's)
          order[j] = l.order[z.row + min(pair * half(z.rows) + r0 + 8 * j, z.rows - 1)];
      };
      if (more) look_up(t);
      for (int i = tile0; ok && more; t = next, more = more_next) {
        const int hx = half(t.rows);
        uint32_t row[kPer];  // in 16-byte pieces; places without a row load row 0, and are not stored
#pragma unroll
        for (int j = 0; j < kPer; ++j) row[j] = (uint32_t)(max(row_of(l, order[j]), 0) * (l.x_stride / 8));
        const uint4* from = reinterpret_cast<const uint4*>(l.x) + (long long)k_lo * S::kSub * 8 + chunk;
        for (int ks = k_lo; ks < k_hi; ++ks, ++it) {
          if (it >= ST && !warp_wait(&c.empty[s], (it / ST - 1) & 1, &c.abort_flag, a.l.status)) {
            ok = false;
            break;
          }
          uint32_t dst = sa(stg + (size_t)s * S::kStage) + 128 * 128 + r0 * 128 + ((chunk ^ r0) << 4);
#pragma unroll
          for (int q = 0; q < S::kSub; ++q, dst += S::kSlab, from += 8) {
            const int bytes = (ks * S::kSub + q) * 64ll + chunk * 8 < l.k ? 16 : 0;  // zeros past K, without a read
#pragma unroll
            for (int j = 0; j < kPer; j += 2)
              if (8 * j < hx) {
#pragma unroll
                for (int z = 0; z < 2; ++z) copy16(dst + (j + z) * 1024, from + row[j + z], bytes);
              }
          }
          copies_arrive(&c.landed[s]);
          s = s + 1 == ST ? 0 : s + 1;
          if (ks == k_lo) {
            more_next = walk.seek(i += step, next);
            if (more_next) look_up(next);
          }
        }
      }
      copies_wait();
    }
    __syncwarp();
  } else {
    const int quarter = warp & 3;
    const uint32_t lanes = tmem + ((uint32_t)(32 * quarter) << 16), run = lanes + 3 * NT;
    Turn<kAccs> acc;
    int waits = 0;
    // the accumulator is full, told by one thread to all
    auto filled = [&] {
      if (threadIdx.x == 0) c.epi_ok[waits & 1] = wait_bar(&c.acc_full[acc.b], acc.par, &c.abort_flag, a.l.status);
      asm volatile("bar.sync 1, 256;" ::: "memory");
      return c.epi_ok[waits++ & 1] != 0;
    };
    auto release = [&] {
      fence_before();
      __syncwarp();
      if (lane == 0) {
        if (CG == 1) mbar_arrive(&c.acc_empty[acc.b]);
        else mbar_arrive_at(peer_addr(sa(&c.acc_empty[acc.b]), first));
      }
      acc.next();
    };
    // a long sum's parts but the last, for `cols` tokens: a warp's lanes and blocks of tokens are its own here and below
    auto add_parts = [&](int cols) {
      for (int k = 1; k < n_parts; ++k) {
        if (!filled()) return false;
        fence_after();
        const uint32_t at = lanes + acc.b * kAcc;
#pragma unroll 1
        for (int n0 = (warp >> 2) * W; n0 < cols; n0 += 2 * W) {
          uint32_t v[W];
          if (k == 1) read_sums(at + n0, 0, 1, v);
          else read_sums(run + n0, at - run, 2, v);
          tmem_st_all<W, 0>(run + n0, v);
        }
        tmem_wait_st();
        release();
      }
      return true;
    };
    if (a.split > 1) {  // one tile; its sums are exchanged below
      if (add_parts(NT)) filled();
    } else {
      Epilogue<W> e(l, sa(stg) + ST * S::kStage + warp * W * 128, lane);
      for (int i = tile0; more; more = walk.seek(i += step, t)) {
        e.start(l.gated ? ((long long)t.n * CG + pair) * 64 + 16 * quarter
                        : ((long long)t.n * CG + pair) * 128 + 32 * quarter,
                t.row, t.group, a.wide);
        auto rows_of = [&](int n0) {  // which of W tokens have a row
          const int left = t.rows - n0;
          const uint32_t in = left >= W ? 0xffffffffu >> (32 - W) : left > 0 ? (1u << left) - 1 : 0u;
          if (!gather) return in;
          return __ballot_sync(kAll, (in >> lane & 1) && source_row(l, t.row + n0 + lane) >= 0);
        };
        int n0 = (warp >> 2) * W;
        uint32_t mask = rows_of(n0);
        if (l.res) e.prefetch(n0, t.rows);
        if (!add_parts(t.rows) || !filled()) break;
        fence_after();
        const uint32_t sums = lanes + acc.b * kAcc;
#pragma unroll 1
        for (; n0 < t.rows; n0 += 2 * W) {
          uint32_t r[W / 4][4];
          if (l.res) e.fetch(n0, mask, r);
          const uint32_t next = rows_of(n0 + 2 * W);
          uint32_t v[W];
          if constexpr (LONG) read_sums(run + n0, sums - run, 2, v);
          else read_sums(sums + n0, NT, n_chains, v);
          __syncwarp();
          e.turn(v);
          __syncwarp();
          with_act(l.act, [&](auto act) {
            if (e.gated) e.template finish<true>(act, n0, mask, r);
            else e.template finish<false>(act, n0, mask, r);
          });
          mask = next;
        }
        release();
      }
    }
    __syncwarp();
  }
  bool failed = false;
  if (CG > 1 || a.split > 1) {
    // a CTA that has given up tells its cluster, which gives a split tile up as one; every
    // thread that raised the flag passes here, and nothing raises it from here on
    if (CG == 1) cluster_wait();
    if (*reinterpret_cast<volatile int*>(&c.abort_flag))
      for (int k = 0; k < team; ++k) store_at(peer_addr(sa(&c.abort_flag), k), 1);
    __syncwarp();
    cluster_sync();
    failed = *reinterpret_cast<volatile int*>(&c.abort_flag);
    // a pair's copies count on its first CTA's barriers, which may have been left by then:
    // a copy takes microseconds, so both CTAs stay half a millisecond
    if (CG > 1 && failed) {
      for (const long long t0 = clock64(); clock64() - t0 < 1000 * 1000;) {
      }
      cluster_sync();
    }
  }
  if (a.split > 1 && !failed) {
    // One tile per cluster (of a dense product), its operands done with everywhere.  Every part
    // lays its sums out in rows and copies each peer the rows that the peer adds up.
    constexpr int kPitch = S::kPitch;
    const int rows_per = 128 / a.split, bytes = rows_per * kPitch * 4;
    float* own = reinterpret_cast<float*>(stg);  // [128][kPitch], then [split - 1][rows_per][kPitch]
    float* in = own + 128 * kPitch;
    if (warp < kEpiWarps) {
      fence_after();
      const int pr = 32 * (warp & 3) + lane;
      const uint32_t acc = tmem + ((uint32_t)(32 * (warp & 3)) << 16), run = acc + 3 * NT;
      const uint32_t last = acc + (n_parts - 1) % 3 * NT;  // of a long sum's parts
#pragma unroll 1
      for (int n0 = (warp >> 2) * W; n0 < NT; n0 += 2 * W) {
        uint32_t v[W];
        if constexpr (LONG) read_sums(run + n0, last - run, 2, v);
        else read_sums(acc + n0, NT, n_chains, v);
#pragma unroll
        for (int i = 0; i < W; i += 4)
          *reinterpret_cast<uint4*>(own + pr * kPitch + n0 + i) = make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
      }
      fence_before();
      fence_async_smem();
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (warp == 0 && elect_one()) {
        mbar_expect(&c.sums, (a.split - 1) * bytes);
        for (int k = 0; k < a.split; ++k) {  // peer k keeps what it gets from part p at p, without itself
          if (k == part) continue;
          const int rank = k * CG + pair, at = part < k ? part : part - 1;
          copy_to_peer(peer_addr(sa(in + at * rows_per * kPitch), rank), own + k * rows_per * kPitch, bytes,
                       peer_addr(sa(&c.sums), rank));
        }
      }
    }
    // the peers' copies are under way to this CTA: no flag ends this wait
    const bool here = drain_bar(&c.sums, 0);
    if (!here && a.l.status) atomicOr(a.l.status, (unsigned long long)MOE_STATUS_TIMEOUT);
    __syncthreads();
    cluster_arrive();  // what the peers copied here has left their shared memory
    walk.start(l, a.shift, 16, a.tn, a.tiles, a.width);
    if (here && walk.seek(tile0, t)) {
      auto sum = [&](int row, int col) {  // a row of this part's, over the parts
        float v = 0.f;
        for (int k = 0; k < a.split; ++k)
          v += k == part ? own[(part * rows_per + row) * kPitch + col]
                         : in[((k < part ? k : k - 1) * rows_per + row) * kPitch + col];
        return v;
      };
      const long long tn = (long long)t.n * CG + pair;
      with_act(l.act, [&](auto act) {
        // neighbouring threads take neighbouring rows: results of one token
        if (l.gated) {
          const int per = rows_per / 2;
          for (int i = threadIdx.x; i < t.rows * per; i += kThreads) {
            const int r = i % per, col = i / per;
            const long long n = tn * 64 + part * per + r;
            if (n >= l.n) continue;
            float g = sum(r / 16 * 32 + r % 16, col), up = sum(r / 16 * 32 + 16 + r % 16, col);
            if (l.bias) g += __bfloat162float(l.bias[n]), up += __bfloat162float(l.bias[l.n + n]);
            finish(l, t.row + col, n, act(g) * up);
          }
        } else {
          for (int i = threadIdx.x; i < t.rows * rows_per; i += kThreads) {
            const int r = i % rows_per, col = i / rows_per;
            const long long n = tn * 128 + part * rows_per + r;
            if (n >= l.n) continue;
            float v = sum(r, col);
            if (l.bias) v += __bfloat162float(l.bias[n]);
            finish(l, t.row + col, n, act(v));
          }
        }
      });
    }
    __syncwarp();
    cluster_wait();  // this CTA's copies have left its shared memory
  }
  fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    fence_after();
    tmem_free<CG>(tmem, S::kCols);
  }
}

// How a product is cut: the kernel's tile, a dense product's tiles of tokens and their width, parts of K.
struct Cut {
  int nt, cg, tiles, width, split;
  long long cost;
};

long long tiles_n(const Linear& l, int cg) {
  const int per = (l.gated ? 64 : 128) * cg;
  return (l.n + (long long)per - 1) / per;
}

// K of a chain at most, in tiles that have room for a long sum.  Groups' tiles of 128 tokens wait for HBM and hide its additions.
int longest(const Linear& l) { return l.f32 || l.offsets ? kPart : kPartBf16; }

template <int NT, int CG, bool LONG>
cudaError_t launch(const Linear& l, const Cut& cut, int sms, cudaStream_t s) {
  using S = Shape<NT, CG>;
  auto kern = linear_kernel<NT, CG, LONG>;
  static Once once;
  cudaError_t e = raise_smem(once, kern, S::kSmem);
  if (e != cudaSuccess) return e;
  Args a{};
  a.l = l;
  const long long tn = tiles_n(l, CG);
  a.shift = NT == 128 ? 7 : 8;  // a dense product is cut beforehand
  a.tiles = cut.tiles;
  a.width = cut.width;
  const long long most = l.offsets ? most_tiles(l, a.shift, tn) : cut.tiles * tn;
  if (most > 0x3fffffff) return cudaErrorInvalidValue;
  a.tn = (int)tn;
  a.nk = (int)((l.k + 64ll * S::kSub - 1) / (64 * S::kSub));
  a.split = cut.split;
  a.part = longest(l) / (64 * S::kSub);
  const int team = CG * a.split;
  auto whole = [&](const void* p, long long stride) {  // 4 results
    return (reinterpret_cast<uintptr_t>(p) & (l.f32 ? 15 : 7)) == 0 && stride % 4 == 0;
  };
  a.wide = whole(l.out, l.out_stride) && whole(l.res, l.res ? l.res_stride : 0);
  CUtensorMap wm, xm{}, xa{};
  e = make_weight_map(&wm, l.w, l.gated, l.k, l.n, l.w_stride * 2, l.groups, l.group_stride * 2);
  if (!l.order) {  // gathered rows need no maps
    if (e == cudaSuccess) e = make_map(&xm, l.x, 2, l.k, l.x_rows, l.x_stride * 2, 32);
    if (e == cudaSuccess) e = make_map(&xa, l.x, 2, l.k, l.x_rows, l.x_stride * 2, S::kX);
  }
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  const long long teams = most < sms / team ? most : sms / team;
  cfg.gridDim = dim3((unsigned)(teams * team));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = S::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {(unsigned)team, 1, 1};
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, wm, xm, xa, a);
}

template <int NT, int CG>
cudaError_t launch(const Linear& l, const Cut& cut, int sms, cudaStream_t s) {
  if constexpr (NT < 256) {
    // of the largest part of K; the smallest is a stage less, two chains at least
    constexpr int kStageK = 64 * Shape<NT, CG>::kSub;
    const long long nk = (l.k + kStageK - 1ll) / kStageK, most = (nk + cut.split - 1) / cut.split;
    if (most * kStageK > (long long)Shape<NT, CG>::kChains * longest(l)) return launch<NT, CG, true>(l, cut, sms, s);
  }
  return launch<NT, CG, false>(l, cut, sms, s);
}

// Parts of K that give every SM a CTA where tiles are few.
int split_for(long long tiles, int nk, int cg, int sms) {
  int s = 1;
  while (2 * s <= kMaxCluster / cg && 2 * s <= nk && tiles * cg * 2 * s <= sms) s *= 2;
  return s;
}

// Estimated cycles of a dense product cut into `tiles` of tokens, kept if less than `best`'s.
template <int NT, int CG>
void consider(const Linear& l, int sms, long long tiles, Cut& best) {
  if (tiles < (l.rows + (long long)NT - 1) / NT || tiles > (l.rows + 15ll) / 16) return;
  const int width = (int)((l.rows + tiles - 1) / tiles + 15) / 16 * 16;
  tiles = (l.rows + (long long)width - 1) / width;
  const long long all = tiles * tiles_n(l, CG);
  constexpr int kSub = Shape<NT, CG>::kSub;
  const int nk = (int)((l.k + 64ll * kSub - 1) / (64 * kSub));  // stages: each part of K has one at least
  // a slab of 64 of K: its MMAs, its copies, the issuing warps' time
  const int mmas = 2 * width, copies = (128 * 128 + (width / CG + 31) / 32 * 4096) / 66, issue = kSub == 2 ? 250 : 400;
  const int slab = mmas > copies ? (mmas > issue ? mmas : issue) : (copies > issue ? copies : issue);
  const int start = CG == 2 && kSub == 2 ? 600 : 0;  // as measured beside the others
  for (int split = 1; split <= split_for(all, nk, CG, sms); split *= 2) {
    const long long per = sms / (CG * split), waves = (all + per - 1) / per;
    const long long cost = waves * ((nk + split - 1) / split) * kSub * slab + width * 40 + start +
                           (split > 1 ? 3000 + 60 * NT : 0);
    if (best.nt == 0 || cost < best.cost) best = {NT, CG, (int)tiles, width, split, cost};
  }
}
template <int NT, int CG>
void consider(const Linear& l, int sms, Cut& best) {
  const long long least = (l.rows + (long long)NT - 1) / NT, tn = tiles_n(l, CG);
  consider<NT, CG>(l, sms, least, best);
  for (int waves = 1; waves <= 3; ++waves) {  // as many as fill the SMs so often
    const long long t = waves * (long long)(sms / CG) / tn;
    if (t > least) consider<NT, CG>(l, sms, t, best);
  }
}

}  // namespace

cudaError_t launch_linear_tc(const Linear& l, int sms, cudaStream_t s) {
  Cut cut{0, 0, 0, 0, 1, 0};
  const bool exact = l.k > (l.f32 ? kPart : kPartBf16);  // tiles of 256 tokens keep one chain
  if (l.offsets) {
    // The rows a group has on average decide; ragged sizes fill either tile as they come.  256 experts, gate and up of
    // 512 x 2,048, 32 / 64 / 128 / 256 rows on average: 148 / 166 / 204 / 283 us in tiles of up to 128 tokens, 161 / 175 /
    // 201 / 254 in tiles of 256 (176 to 830 in lone CTAs' of 32, which tie below 8 rows).
    if (l.rows / l.groups < 100 || exact) return launch<128, 2>(l, cut, sms, s);
    return launch<256, 2>(l, cut, sms, s);
  }
  consider<32, 1>(l, sms, cut);
  consider<128, 1>(l, sms, cut);
  consider<128, 2>(l, sms, cut);
  if (!exact) consider<256, 2>(l, sms, cut);
  if (cut.nt == 128 && cut.cg == 2) return launch<128, 2>(l, cut, sms, s);
  if (cut.nt == 32) return launch<32, 1>(l, cut, sms, s);
  if (cut.nt == 128) return launch<128, 1>(l, cut, sms, s);
  return launch<256, 2>(l, cut, sms, s);
}

}  // namespace moe

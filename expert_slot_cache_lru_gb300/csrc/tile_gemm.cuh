// tile_gemm.cuh -- out = P Q^T on the tensor cores for K-major matrices of bf16
// or block-scaled 4-bit elements: the router's logits and the 4-bit product.
//
// A tile is 128 rows of P (256 with a CTA pair, CG = 2) times NT rows of Q;
// sums are fp32 in tensor memory.  A stage of the pipeline is 128 bytes of every
// row: 64 bf16 or 256 4-bit elements, four MMAs.  CTAs (or pairs) are persistent
// and take tiles in turn.  Warps of a CTA:
//   0..7   epilogue: tensor memory -> registers -> global scales -> out.  Warp w
//          reads lanes 32 (w % 4) .., half w / 4 of the columns; 4-bit kinds alternate
//          two accumulators, so the next tile's MMAs run beside it;
//   8..15  block scales (4-bit kinds), shared memory -> tensor memory in the order
//          the MMA reads, two groups of four warps on alternate stages (one group alone
//          left the MMAs of an 8,192 x 8,192 x 4,096 product waiting: 150 us).
//          (tcgen05.cp would copy them too, but measured 52 cycles per 512 bytes in
//          series with the MMAs.)
//   16..23 block scales, global -> shared memory, 64 bytes of a row at a time: TMA
//          where the banks' rows are whole 16-byte pieces (K a multiple of 256 or 512),
//          else aligned loads, shifted;
//   then   one warp of TMA loads of the operands, one of MMAs (the first CTA's of a pair).
// A pair halves what each SM takes in of Q: an SM takes in about 64 bytes per
// cycle, which bounds the bf16 tiles and a lone CTA's 4-bit ones.
// Scale order: the 32-bit word of row r and K step j belongs in lane r % 32 of
// every warp's quarter, column r / 32 of block j.  NVFP4: a word is the four
// scales of one 64-element step; MXFP4: the two scales of two steps, picked by
// the instruction's scale ids.
// Where tiles are few, `split` CTAs (pairs) of a cluster share a tile: each sums
// its part of K and then, through distributed shared memory, its part of the
// tile's results over the parts in ascending order.
// Every wait is bounded; on a timeout the CTA reports it, drains its copies and
// MMAs, frees its tensor memory and returns.  A cluster gives a split tile up as one:
// a tile is stored whole and right or not at all.
#pragma once

#include <cuda_bf16.h>

#include "tc.cuh"

namespace moe {
namespace tg {

using namespace tc;

enum Kind { kBf16, kNv, kMx };

constexpr int kEpiWarps = 8, kScaleWarp = 8, kCopyWarp = 16;
constexpr int kGroups = 2;  // groups of scales in shared memory, 64 bytes of each row
// CTAs of a cluster: eights do not all find room at once (128 CTAs in eights
// started up to 6 us apart)
constexpr int kMaxCluster = 4;

template <Kind KIND, int NT, int CG>
struct Shape {
  static constexpr int kQ = NT / CG;                          // Q rows a CTA loads
  static constexpr int kBlocks = KIND == kNv ? 4 : KIND == kMx ? 2 : 0;  // scale words per row and stage
  static constexpr int kTmaWarp = kBlocks ? 24 : kEpiWarps, kMmaWarp = kTmaWarp + 1;
  static constexpr int kThreads = 32 * (kMmaWarp + 1);
  static constexpr int kPer = KIND == kMx ? 2 : 1;            // stages in 16 bytes of a row's scales
  static constexpr int kGroupStages = 4 * kPer;
  static constexpr int kQRows = (NT + 31) / 32 * 32;          // Q rows of scales in shared memory
  static constexpr int kQCols = NT < 128 ? 4 : (NT + 31) / 32;  // Q columns of a scale block
  static constexpr int kScaleCols = kBlocks * (4 + kQCols);   // of tensor memory, per stage
  static constexpr int kStage = 128 * 128 + kQ * 128;
  static constexpr int kSlot = (128 + kQRows) * 64;           // a group of scales
  static constexpr int kScaleSmem = kBlocks ? kGroups * kSlot : 0;
  static constexpr int kOut = NT < 64 ? 0 : kEpiWarps * 4096;  // results on their way out
  static constexpr int kFit = (226 * 1024 - 1024 - 1024 - kScaleSmem - kOut) / kStage;
  static constexpr int kStages = kFit > 12 ? 12 : kFit;
  // stages of scales in tensor memory
  static constexpr int kBufs = !kBlocks ? 1 : 2 * NT + 4 * kScaleCols <= 512 ? 4 : 3;
  // Sums of a tile: the tensor cores add with truncation, an error that grows with the
  // chain of additions, so bf16 tiles use the tensor memory for up to four parts of
  // K, added up in the epilogue; 4-bit tiles (chains four times shorter) alternate two tiles.
  static constexpr int kChains = kBlocks ? 1 : 512 / NT < 4 ? 512 / NT : 4;
  static constexpr int kAcc = kBlocks && 2 * NT + kBufs * kScaleCols <= 512 ? 2 : 1;
  static constexpr int kUsed = kAcc * kChains * NT + kBufs * kScaleCols;
  static constexpr int kCols = kUsed <= 32 ? 32 : kUsed <= 64 ? 64 : kUsed <= 128 ? 128 : kUsed <= 256 ? 256 : 512;
  static constexpr int kSmem = kStages * kStage + kOut + kScaleSmem + 1024;
  static_assert(kUsed <= 512 && kStage % 1024 == 0 && kStages >= kBufs, "tile shape");
  static_assert(kStages * kStage + kOut >= 128 * (NT + 4) * 4 * (CG == 1 ? 7 : 6) / 4, "room for a split's sums");
};

struct Args {
  const uint8_t *ps, *qs;  // scale banks
  int p_rows, q_rows;
  int tiles_p, tiles_q;
  int nk;                  // stages of K
  int sb;                  // scale bytes per row
  int tma_scales;          // the scale banks' rows are whole 16-byte pieces
  int split;               // parts of K
  const float *g0, *g1;
  void* out;
  long long out_stride;
  int f32;
  int wide;                // the output's rows are whole 16-byte pieces
  unsigned long long* status;
};

template <int ST>
struct Ctl {
  uint64_t full[ST], empty[ST], scaled[4], rows_full[kGroups], rows_empty[kGroups];
  uint64_t acc_full[2], acc_empty[2], drain, sums;
  uint32_t tmem;
  int abort_flag, epi_ok[2];  // epi_ok: the epilogue's wait, by tile parity
};

// tiles in strips of 8 P tiles, so that concurrent CTAs share operands in L2
__device__ __forceinline__ void tile_at(const Args& a, int t, int& tp, int& tq) {
  const int per = 8 * a.tiles_q, g = t / per, r = t - g * per;
  const int n = min(8, a.tiles_p - g * 8);
  tp = g * 8 + r % n;
  tq = r / n;
}

// 16 aligned bytes at the end of a bank of `bytes` bytes (nothing past it is read)
static __device__ __noinline__ uint4 bank_word(const uint8_t* bank, long long bytes, long long word) {
  uint32_t w[4] = {0, 0, 0, 0};
  for (int j = 0; j < 16 && word * 16 + j < bytes; ++j)
    w[j >> 2] |= (uint32_t)bank[word * 16 + j] << (8 * (j & 3));
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// bytes sh .. sh + 15 of two neighbouring words, those from `n` on zero
__device__ __forceinline__ uint4 cut(uint4 a, uint4 b, int sh, int n) {
  uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  if (sh & 8) {
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  }
  if (sh & 4) {
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  }
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    o[i] = __funnelshift_r(w[i], w[i + 1], 8 * (sh & 3));
    const int left = n - 4 * i;  // bytes to keep
    o[i] = left >= 4 ? o[i] : left <= 0 ? 0u : o[i] & (0xffffffffu >> (32 - 8 * left));
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}
// A group of block scales of a tile into shared memory where the banks' rows are not
// whole 16-byte pieces: 64 bytes from `off` of 128 P rows and NT Q rows, zeros beyond the
// matrix, in the 64-byte swizzle of a TMA copy.  256 threads, four per row; the loads
// wait in registers for the slot they go to.
template <int NT>
struct ScaleRows {
  static constexpr int PR = 2, QR = (NT + 63) / 64;  // rows per thread, 64 apart
  uint4 w0[PR + QR], w1[PR + QR];
  int sh[PR + QR], n;
  __device__ __forceinline__ void load(const Args& a, int p_row, int q_row, int off, int tid);
  __device__ __forceinline__ void store(uint8_t* dst, int tid) const;
};
template <int NT>
__device__ __forceinline__ void ScaleRows<NT>::load(const Args& a, int p_row, int q_row, int off, int tid) {
  const int at = off + 16 * (tid & 3), r0 = tid >> 2;
  n = min(16, a.sb - at);
#pragma unroll
  for (int u = 0; u < PR + QR; ++u) {
    const bool is_p = u < PR;
    const int rows = is_p ? a.p_rows : a.q_rows;
    // past 2^31 - 1 a row is negative, and not below `rows` without sign
    const int row = (int)((unsigned)(is_p ? p_row : q_row) + (unsigned)(is_p ? 64 * u : 64 * (u - PR)) + r0);
    const uint8_t* bank = is_p ? a.ps : a.qs;
    const long long bytes = (long long)rows * a.sb, byte = (long long)row * a.sb + at;
    w0[u] = w1[u] = make_uint4(0, 0, 0, 0);
    sh[u] = (int)(byte & 15);
    if ((unsigned)row < (unsigned)rows && n > 0 && (is_p || r0 + 64 * (u - PR) < NT)) {
      if (((byte >> 4) + 2) * 16 <= bytes) {  // else at the bank's end
        w0[u] = reinterpret_cast<const uint4*>(bank)[byte >> 4];
        w1[u] = reinterpret_cast<const uint4*>(bank)[(byte >> 4) + 1];
      } else {
        w0[u] = bank_word(bank, bytes, byte >> 4);
        w1[u] = bank_word(bank, bytes, (byte >> 4) + 1);
      }
    }
  }
}
template <int NT>
__device__ __forceinline__ void ScaleRows<NT>::store(uint8_t* dst, int tid) const {
  const int chunk = tid & 3, r0 = tid >> 2;
#pragma unroll
  for (int u = 0; u < PR + QR; ++u) {
    const int r = u < PR ? r0 + 64 * u : 128 + r0 + 64 * (u - PR);
    if (r < 128 + NT)
      *reinterpret_cast<uint4*>(dst + r * 64 + ((chunk ^ ((r >> 1) & 3)) << 4)) = cut(w0[u], w1[u], sh[u], n);
  }
}

// Instruction descriptors: K-major operands, fp32 sums.  4 bits: e2m1 x e2m1, K 64, scales
// e4m3 or e8m0, `id` the scale bytes of a word; bf16: K 16.
template <Kind KIND>
__device__ __forceinline__ uint32_t idesc(int m, int n, int id) {
  const uint32_t mn = ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
  if (KIND == kBf16) return mn | (1u << 4) | (1u << 7) | (1u << 10);
  return mn | ((uint32_t)id << 4) | (1u << 7) | (1u << 10) | (KIND == kNv ? 0u : 1u << 23) |
         ((uint32_t)id << 29);
}
#define MOE_TG_MMA4(cg, kind, vec)                                                              \
  asm volatile(                                                                                 \
      "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"                                             \
      " tcgen05.mma.cta_group::" cg ".kind::" kind ".block_scale.scale_vec::" vec               \
      " [%0], %1, %2, %3, [%4], [%5], p;\n}\n" ::"r"(d),                                        \
      "l"(p), "l"(q), "r"(id), "r"(sp), "r"(sq), "r"(acc)                                       \
      : "memory")
#define MOE_TG_MMA16(cg)                                                                        \
  asm volatile(                                                                                 \
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"                                             \
      " tcgen05.mma.cta_group::" cg ".kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),            \
      "l"(p), "l"(q), "r"(id), "r"(acc)                                                         \
      : "memory")
template <Kind KIND, int CG>
__device__ __forceinline__ void mma(uint32_t d, uint64_t p, uint64_t q, uint32_t id, uint32_t sp,
                                    uint32_t sq, uint32_t acc) {
  if constexpr (KIND == kBf16) {
    if constexpr (CG == 1) MOE_TG_MMA16("1");
    else MOE_TG_MMA16("2");
  } else if constexpr (KIND == kNv) {
    if constexpr (CG == 1) MOE_TG_MMA4("1", "mxf4nvf4", "4X");
    else MOE_TG_MMA4("2", "mxf4nvf4", "4X");
  } else {
    if constexpr (CG == 1) MOE_TG_MMA4("1", "mxf4", "2X");
    else MOE_TG_MMA4("2", "mxf4", "2X");
  }
}
#undef MOE_TG_MMA4
#undef MOE_TG_MMA16

__device__ __forceinline__ void store_one(const Args& a, long long at, float v) {
  if (a.f32) static_cast<float*>(a.out)[at] = v;
  else static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(v);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float global_scale(const Args& a) {
  return (a.g0 ? *a.g0 : 1.f) * (a.g1 ? *a.g1 : 1.f);
}

// W columns of the warp's lanes, the sums of n_chains parts of K added up in order
template <int NT, int W>
__device__ __forceinline__ void read_sums(uint32_t at, int n_chains, uint32_t (&v)[W]) {
  uint32_t u[W];
  tmem_ld(at, v);
  if (n_chains > 1) tmem_ld(at + NT, u);
  tmem_wait_ld();
  for (int k = 1; k < n_chains; ++k) {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) + __uint_as_float(u[i]));
    if (k + 1 < n_chains) {
      tmem_ld(at + (k + 1) * NT, u);
      tmem_wait_ld();
    }
  }
}

// The end of a split tile: `rows` rows of this part and `cols` columns, S parts' sums of
// each added up in order and stored, four neighbouring columns per thread; several
// loads in flight, since little else hides their latency here.
// own: this part's sums [128][pitch]; in: the other parts' [S - 1][rows_per][pitch].
template <int NT, int S>
__device__ __forceinline__ void add_parts(const Args& a, uint32_t own, uint32_t in, int part, int rows,
                                          int cols, long long to0, float g, int threads) {
  constexpr int kPitch = NT + 4, kRows = 128 / S, U = 8 / S;
  for (int i0 = threadIdx.x; i0 < rows * (NT / 4); i0 += U * threads) {
    float4 x[U][S];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = min(i0 + u * threads, rows * (NT / 4) - 1), row = i / (NT / 4), col = i % (NT / 4) * 4;
#pragma unroll
      for (int k = 0; k < S; ++k)
        x[u][k] = lds4(k == part ? own + 4 * ((part * kRows + row) * kPitch + col)
                                 : in + 4 * (((k < part ? k : k - 1) * kRows + row) * kPitch + col));
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * threads, row = i / (NT / 4), col = i % (NT / 4) * 4;
      if (i >= rows * (NT / 4) || col >= cols) continue;
      float4 v = x[u][0];
#pragma unroll
      for (int k = 1; k < S; ++k) v.x += x[u][k].x, v.y += x[u][k].y, v.z += x[u][k].z, v.w += x[u][k].w;
      const long long to = to0 + row * a.out_stride + col;
      const float r[4] = {v.x * g, v.y * g, v.z * g, v.w * g};
      if (a.wide && col + 4 <= cols) {
        if (a.f32)
          *reinterpret_cast<float4*>(static_cast<float*>(a.out) + to) = make_float4(r[0], r[1], r[2], r[3]);
        else
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + to) =
              make_uint2(pack2(r[0], r[1]), pack2(r[2], r[3]));
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (col + j < cols) store_one(a, to + j, r[j]);
      }
    }
  }
}

// SWAP: out[q][p] (P the weights, Q the tokens); else out[p][q].
template <Kind KIND, int NT, int CG, bool SWAP>
__global__ void __launch_bounds__(Shape<KIND, NT, CG>::kThreads, 1)
gemm_kernel(const __grid_constant__ CUtensorMap pmap, const __grid_constant__ CUtensorMap qmap,
            const __grid_constant__ CUtensorMap psmap, const __grid_constant__ CUtensorMap qsmap,
            const __grid_constant__ CUtensorMap omap, const Args a) {
  using T = Shape<KIND, NT, CG>;
  constexpr int ST = T::kStages, kThreads = T::kThreads;
  extern __shared__ uint8_t raw[];
  uint8_t* stg = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint8_t* ostg = stg + (size_t)ST * T::kStage;
  uint8_t* sstg = ostg + T::kOut;
  __shared__ Ctl<ST> c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int W = NT < 64 ? 16 : 32;  // columns the epilogue reads at a time
  // cluster: `split` parts of K, each CG CTAs; a lone CTA's cluster is itself
  const int crank = CG == 1 && a.split == 1 ? 0 : (int)cluster_rank();
  const int pair = crank % CG, first = crank - pair, part = crank / CG;
  const int team = CG * a.split;
  // a part of K starts at a whole 16 bytes of scales
  const int nkp = (a.nk + T::kPer - 1) / T::kPer;
  const int k_lo = nkp * part / a.split * T::kPer,
            k_hi = min(a.nk, nkp * (part + 1) / a.split * T::kPer), n_k = k_hi - k_lo;
  const int n_tiles = a.tiles_p * a.tiles_q, tile0 = blockIdx.x / team, step = gridDim.x / team;
  const int n_chains = min(T::kChains, n_k);
  const uint16_t mask = (uint16_t)(((1 << CG) - 1) << first);

  pdl_trigger();
  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&c.full[i], 1);
      mbar_init(&c.empty[i], 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&c.scaled[i], 4 * CG);
    for (int i = 0; i < kGroups; ++i) {
      mbar_init(&c.rows_full[i], a.tma_scales ? 1 : 256);
      mbar_init(&c.rows_empty[i], 8);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c.acc_full[i], 1);
      mbar_init(&c.acc_empty[i], kEpiWarps * CG);
    }
    mbar_init(&c.drain, 1);
    mbar_init(&c.sums, 1);
    c.abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == T::kMmaWarp) tmem_alloc<CG>(&c.tmem, T::kCols);
  fence_before();
  __syncthreads();
  if (CG > 1) cluster_sync();  // the peer's barriers exist before anything arrives there
  else if (a.split > 1) cluster_arrive();  // waited for before anything goes to a peer
  fence_after();
  const uint32_t tmem = c.tmem;
  pdl_wait();

  if (warp == T::kTmaWarp) {
    int it = 0, s = 0;
    bool ok = true;
    for (int t = tile0; t < n_tiles && ok; t += step) {
      int tp, tq;
      tile_at(a, t, tp, tq);
      for (int ks = k_lo; ks < k_hi; ++ks, ++it) {
        if (it >= ST && !warp_wait(&c.empty[s], (it / ST - 1) & 1, &c.abort_flag, a.status)) {
          ok = false;
          break;
        }
        if (elect_one()) {
          uint8_t* p = stg + (size_t)s * T::kStage;
          const int x = ks * (KIND == kBf16 ? 64 : 128);
          // a pair's copies all count on the first CTA's barrier
          if (pair == 0) mbar_expect(&c.full[s], CG * T::kStage);
          const uint32_t bar = CG == 1 ? sa(&c.full[s]) : peer_addr(sa(&c.full[s]), first);
          tma_load<CG>(p, &pmap, x, (tp * CG + pair) * 128, bar);
          tma_load<CG>(p + 128 * 128, &qmap, x, tq * NT + pair * T::kQ, bar);
        }
        __syncwarp();
        s = s + 1 == ST ? 0 : s + 1;
      }
    }
    // the copies in flight land before the CTA ends, whichever warp may have given up
    if (pair == 0)
      for (int i = it > ST ? it - ST : 0; i < it; ++i)
        if (!drain_bar(&c.full[i % ST], (i / ST) & 1)) break;
    __syncwarp();
  } else if (warp == T::kMmaWarp) {
    if (pair == 0) {
      int u = 0, s = 0, sbuf = 0;
      uint32_t full_par = 0, scaled_par = 0;  // parities of this round through the rings
      bool ok = true;
      const uint64_t p_base = desc_tile(sa(stg)), q_base = desc_tile(sa(stg) + 128 * 128);
      for (int t = tile0; t < n_tiles && ok; t += step, ++u) {
        const int b = u % T::kAcc;
        if (u >= T::kAcc &&
            !warp_wait(&c.acc_empty[b], (u / T::kAcc - 1) & 1, &c.abort_flag, a.status))
          break;
        uint32_t d = tmem + b * NT;
        int chain = 0, first_of = 0;  // the part of K being summed, its first stage
        for (int i = 0; i < n_k; ++i) {
          if (T::kChains > 1 && i == n_k * (chain + 1) / n_chains) {
            ++chain;
            first_of = i;
            d += NT;
          }
          // both at once; one after the other only if one is not there yet
          const bool there = mbar_test(&c.full[s], full_par) &
                             (!T::kBlocks || mbar_test(&c.scaled[sbuf], scaled_par));
          if (!__all_sync(0xffffffffu, there) &&
              ((T::kBlocks && !warp_wait(&c.scaled[sbuf], scaled_par, &c.abort_flag, a.status)) ||
               !warp_wait(&c.full[s], full_par, &c.abort_flag, a.status))) {
            ok = false;
            break;
          }
          fence_after();
          if (elect_one()) {
            const uint64_t p0 = p_base + (uint64_t)(s * (T::kStage / 16)),
                           q0 = q_base + (uint64_t)(s * (T::kStage / 16));
            const uint32_t cp = tmem + T::kAcc * NT + sbuf * T::kScaleCols, cq = cp + 4 * T::kBlocks;
#pragma unroll
            for (int j = 0; j < 4; ++j) {  // 32 bytes of every row each
              const int w = KIND == kMx ? j / 2 : j, id = KIND == kMx ? 2 * (j & 1) : 0;
              mma<KIND, CG>(d, p0 + 2 * j, q0 + 2 * j, idesc<KIND>(128 * CG, NT, id), cp + 4 * w,
                            cq + T::kQCols * w, j > 0 || i > first_of);
            }
            mma_commit<CG>(&c.empty[s], mask);
          }
          __syncwarp();
          if (++s == ST) s = 0, full_par ^= 1;
          if (++sbuf == T::kBufs) sbuf = 0, scaled_par ^= 1;
        }
        if (!ok) break;
        if (elect_one()) mma_commit<CG>(&c.acc_full[b], mask);
        __syncwarp();
      }
      if (elect_one()) mma_commit<CG>(&c.drain, mask);
      __syncwarp();
    }
    drain_bar(&c.drain, 0);  // every MMA has finished before the tensor memory is freed
    __syncwarp();
  } else if (warp >= kCopyWarp) {
    if constexpr (T::kBlocks > 0) {
      const int n_warps = a.tma_scales ? 1 : 8;  // one lane of TMA, or all 256 threads
      unsigned group = 0;
      bool ok = warp - kCopyWarp < n_warps;
      for (int t = tile0; t < n_tiles && ok; t += step) {
        int tp, tq;
        tile_at(a, t, tp, tq);
        const int p_row = (tp * CG + pair) * 128, q_row = tq * NT;
        // groups start at the first stage of the tile's part of K
        for (int ks = k_lo; ks < k_hi; ks += T::kGroupStages, ++group) {
          const unsigned slot = group % kGroups;
          const int off = ks * (16 / T::kPer), tid = threadIdx.x - 32 * kCopyWarp;
          ScaleRows<NT> rows;
          if (!a.tma_scales) rows.load(a, p_row, q_row, off, tid);
          if (group >= kGroups && !warp_wait(&c.rows_empty[slot], (group / kGroups - 1) & 1,
                                             &c.abort_flag, a.status)) {
            ok = false;
            break;
          }
          uint8_t* dst = sstg + slot * T::kSlot;
          if (a.tma_scales) {
            if (elect_one()) {
              mbar_expect(&c.rows_full[slot], (128 + NT) * 64);
              tma_load<1>(dst, &psmap, off, p_row, sa(&c.rows_full[slot]));
              tma_load<1>(dst + 128 * 64, &qsmap, off, q_row, sa(&c.rows_full[slot]));
            }
            __syncwarp();
          } else {
            rows.store(dst, tid);
            mbar_arrive(&c.rows_full[slot]);
          }
        }
      }
      if (warp == kCopyWarp && a.tma_scales)  // as the operands' copies
        for (unsigned i = group > kGroups ? group - kGroups : 0; i < group; ++i)
          if (!drain_bar(&c.rows_full[i % kGroups], (i / kGroups) & 1)) break;
    }
    __syncwarp();
  } else if (warp >= kScaleWarp) {
    if constexpr (T::kBlocks > 0) {
      const uint32_t quarter = (uint32_t)(32 * (warp & 3)) << 16;
      const unsigned mine = (warp - kScaleWarp) >> 2;  // takes the stages of this parity
      unsigned it = 0, group = 0;
      bool ok = true;
      for (int t = tile0; t < n_tiles && ok; t += step) {
        for (int ks = k_lo; ks < k_hi && ok; ks += T::kGroupStages, ++group) {
          const unsigned slot = group % kGroups, m = min(T::kGroupStages, k_hi - ks);
          if (!warp_wait(&c.rows_full[slot], (group / kGroups) & 1, &c.abort_flag, a.status)) {
            ok = false;
            break;
          }
#pragma unroll 1
          for (unsigned x = (it ^ mine) & 1; x < m; x += 2) {
            const unsigned n = it + x, buf = n % T::kBufs;
            // lane's rows, lane + 32 q: word j of row q belongs in column q of block j
            const uint8_t* sp = sstg + slot * T::kSlot + lane * 64 +
                                (((x / T::kPer) ^ ((lane >> 1) & 3)) << 4) +
                                (KIND == kMx ? 8 * (x & 1) : 0);
            uint32_t w[T::kScaleCols];
#pragma unroll
            for (int q = 0; q < 4 + T::kQCols; ++q) {
              uint32_t v[4] = {0, 0, 0, 0};
              if (q < 4 || 32 * (q - 4) < T::kQRows) {
                if constexpr (KIND == kNv) {
                  const uint4 u = *reinterpret_cast<const uint4*>(sp + 2048 * q);
                  v[0] = u.x, v[1] = u.y, v[2] = u.z, v[3] = u.w;
                } else {
                  const uint2 u = *reinterpret_cast<const uint2*>(sp + 2048 * q);
                  v[0] = u.x, v[1] = u.y;
                }
              }
#pragma unroll
              for (int j = 0; j < T::kBlocks; ++j)
                w[q < 4 ? 4 * j + q : 4 * T::kBlocks + T::kQCols * j + q - 4] = v[j];
            }
            // a buffer's previous scales have been used once MMA n - kBufs is done
            if (n >= T::kBufs) {
              const unsigned was = n - T::kBufs;
              if (!warp_wait(&c.empty[was % ST], (was / ST) & 1, &c.abort_flag, a.status)) {
                ok = false;
                break;
              }
            }
            fence_after();
            tmem_st_all(tmem + quarter + T::kAcc * NT + buf * T::kScaleCols, w);
            tmem_wait_st();
            fence_before();
            __syncwarp();
            if (lane == 0) {
              if (CG == 1) mbar_arrive(&c.scaled[buf]);
              else mbar_arrive_at(peer_addr(sa(&c.scaled[buf]), first));
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&c.rows_empty[slot]);
          it += m;
        }
      }
    }
    __syncwarp();
  } else {
    const float g = global_scale(a);
    int u = 0, piece = 0;
    for (int t = tile0; t < n_tiles; t += step, ++u) {
      const int b = u % T::kAcc;
      int tp, tq;
      tile_at(a, t, tp, tq);
      if (threadIdx.x == 0)
        c.epi_ok[u & 1] = wait_bar(&c.acc_full[b], (u / T::kAcc) & 1, &c.abort_flag, a.status);
      asm volatile("bar.sync 1, 256;" ::: "memory");
      if (!c.epi_ok[u & 1] || a.split > 1) break;  // a split's sums are exchanged below
      fence_after();
      const int pr = 32 * (warp & 3) + lane;
      const uint32_t acc = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + b * NT;
      const long long p = ((long long)tp * CG + pair) * 128 + pr;
      // a warp whose rows are all past the matrix has nothing to stage: its output buffers
      // may still be under a copy, which a piece without a copy of its own would not wait for
      const int n_end = p - lane < a.p_rows ? NT : 0;
#pragma unroll 1
      for (int n0 = (warp >> 2) * W; n0 < n_end; n0 += 2 * W) {
        const long long q0 = (long long)tq * NT + n0;
        if (q0 >= a.q_rows) break;
        uint32_t v[W];
        read_sums<NT>(acc + n0, n_chains, v);
        const int nq = (int)(a.q_rows - q0 < W ? a.q_rows - q0 : W);
        if (SWAP) {
          if (p < a.p_rows) {
#pragma unroll
            for (int i = 0; i < W; ++i)
              if (i < nq) store_one(a, (q0 + i) * a.out_stride + p, __uint_as_float(v[i]) * g);
          }
        } else if (a.wide) {
          // through shared memory (the copy's swizzle) and out by TMA, 32 rows x 32
          // columns per warp: lanes that store their own rows touch 32 lines a store and
          // keep the block scales waiting (8,192 x 8,192 x 4,096: 100 us, so 94)
          if constexpr (!SWAP) {
            uint8_t* o = ostg + warp * 4096 + (a.f32 ? 0 : (piece & 1) * 2048);
            if (lane == 0) {  // what this buffer held has been read (bf16: two buffers in turn)
              if (a.f32) store_wait_read<0>();
              else store_wait_read<1>();
            }
            __syncwarp();
            if (a.f32) {
#pragma unroll
              for (int i = 0; i < 8; ++i)
                *reinterpret_cast<float4*>(o + lane * 128 + ((i ^ (lane & 7)) << 4)) =
                    make_float4(__uint_as_float(v[4 * i]) * g, __uint_as_float(v[4 * i + 1]) * g,
                                __uint_as_float(v[4 * i + 2]) * g, __uint_as_float(v[4 * i + 3]) * g);
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  w[j] = pack2(__uint_as_float(v[8 * i + 2 * j]) * g, __uint_as_float(v[8 * i + 2 * j + 1]) * g);
                *reinterpret_cast<uint4*>(o + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4)) =
                    make_uint4(w[0], w[1], w[2], w[3]);
              }
            }
            fence_async_smem();
            __syncwarp();
            if (lane == 0) tma_store(&omap, o, (int)q0, (int)p);  // rows past the matrix are not written
            ++piece;  // one copy each: the waits above count copies
          }
        } else {  // other row lengths: turned in shared memory, so that a row's lanes are neighbours
          if constexpr (!SWAP) {
            float* o = reinterpret_cast<float*>(ostg + warp * 4096);
            __syncwarp();
#pragma unroll
            for (int i = 0; i < W; ++i) o[lane * 32 + (i ^ lane)] = __uint_as_float(v[i]) * g;
            __syncwarp();
            const int rows = (int)min(32LL, a.p_rows - (p - lane));
            for (int r = 0; r < rows; ++r)
              if (lane < nq) store_one(a, (p - lane + r) * a.out_stride + q0 + lane, o[r * 32 + (lane ^ r)]);
          }
        }
      }
      fence_before();
      __syncwarp();
      if (lane == 0) {
        if (CG == 1) mbar_arrive(&c.acc_empty[b]);
        else mbar_arrive_at(peer_addr(sa(&c.acc_empty[b]), first));
      }
    }
    if (lane == 0) store_wait_done();
    __syncwarp();
  }
  bool failed = false;
  if (CG > 1 || a.split > 1) {
    // a CTA that has given up tells its cluster, which gives the tile up as one; every
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
    // One tile per cluster, its operands done with everywhere.  Every part lays its
    // sums out in rows and copies each peer the rows that the peer adds up; stores
    // to the peers one by one took 3,000 cycles of a 128 x 128 tile.
    constexpr int kPitch = NT + 4;  // rows 4 banks apart
    const int rows_per = 128 / a.split, bytes = rows_per * kPitch * 4;
    float* own = reinterpret_cast<float*>(stg);  // [128][kPitch], then [split - 1][rows_per][kPitch]
    float* in = own + 128 * kPitch;
    if (warp < kEpiWarps) {
      fence_after();
      const int pr = 32 * (warp & 3) + lane;
      const uint32_t acc = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
#pragma unroll 1
      for (int n0 = (warp >> 2) * W; n0 < NT; n0 += 2 * W) {
        uint32_t v[W];
        read_sums<NT>(acc + n0, n_chains, v);
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
    if (!here && a.status) atomicOr(a.status, (unsigned long long)MOE_STATUS_TIMEOUT);
    __syncthreads();
    cluster_arrive();  // what the peers copied here has left their shared memory
    int tp, tq;
    tile_at(a, tile0, tp, tq);
    const float g = global_scale(a);
    const long long p0 = ((long long)tp * CG + pair) * 128 + part * rows_per, q0 = (long long)tq * NT;
    const int rows = (int)max(0LL, min((long long)rows_per, a.p_rows - p0));
    const int cols = (int)min((long long)NT, a.q_rows - q0);
    if (!here) {
    } else if (SWAP) {  // neighbouring threads take neighbouring rows: outputs of one token
      for (int i = threadIdx.x; i < cols * rows_per; i += kThreads) {
        const int row = i % rows_per, col = i / rows_per;
        float v = 0.f;
        for (int k = 0; k < a.split; ++k)
          v += k == part ? own[(part * rows_per + row) * kPitch + col]
                         : in[((k < part ? k : k - 1) * rows_per + row) * kPitch + col];
        if (row < rows) store_one(a, (q0 + col) * a.out_stride + p0 + row, v * g);
      }
    } else if (a.split == 2) {
      add_parts<NT, 2>(a, sa(own), sa(in), part, rows, cols, p0 * a.out_stride + q0, g, kThreads);
    } else {
      add_parts<NT, 4>(a, sa(own), sa(in), part, rows, cols, p0 * a.out_stride + q0, g, kThreads);
    }
    __syncwarp();
    cluster_wait();  // this CTA's copies have left its shared memory
  }
  fence_before();
  __syncthreads();
  if (warp == T::kMmaWarp) {
    fence_after();
    tmem_free<CG>(tmem, T::kCols);
  }
}

// What a caller fills in: the matrices and the output.
struct Problem {
  const void *p, *q;           // K-major rows; p_stride, q_stride bytes apart
  long long p_stride, q_stride;
  int p_rows, q_rows, k;
  const uint8_t *ps, *qs;      // scale banks (4-bit kinds)
  const float *g0, *g1;
  void* out;
  long long out_stride;
  bool f32;
  unsigned long long* status;
};

// Parts of K that give every SM a CTA where tiles are few.
inline int split_for(long long tiles, int nk, int cg, int sms) {
  int s = 1;
  while (2 * s <= kMaxCluster / cg && 2 * s <= nk && tiles * cg * 2 * s <= sms) s *= 2;
  return s;
}

// Estimated cycles of a product with this tile, the measure the tile is chosen by:
// stages times the cycles one was measured to take when nothing else bounds it (an SM
// takes in about 64 bytes per cycle; a stage of 4-bit rows has its scales to move), and a
// split's exchange of partial sums (2,500 cycles and 18 bytes per cycle).
template <Kind KIND, int NT, int CG>
long long cycles(long long p_rows, long long q_rows, int k, int sms) {
  using T = Shape<KIND, NT, CG>;
  constexpr int kStageCycles = KIND == kBf16 ? (NT <= 64 ? 450 : NT <= 128 ? 494 : 520)
                                             : (NT <= 64 ? 480 : NT <= 128 ? 600 : 630);
  const long long tiles = (p_rows + 128 * CG - 1) / (128 * CG) * ((q_rows + NT - 1) / NT);
  const int slab = KIND == kBf16 ? 64 : 256, nk = (int)((k + (long long)slab - 1) / slab);
  const int split = split_for(tiles, (nk + T::kPer - 1) / T::kPer, CG, sms);
  const long long per = sms / (CG * split), waves = (tiles + per - 1) / per;
  return waves * ((nk + split - 1) / split * kStageCycles) + (split > 1 ? 2500 + 128 * NT * 4 / 18 : 0);
}

template <Kind KIND, int NT, int CG, bool SWAP>
cudaError_t launch(const Problem& l, int sms, cudaStream_t s) {
  using T = Shape<KIND, NT, CG>;
  auto kern = gemm_kernel<KIND, NT, CG, SWAP>;
  static Once once;
  cudaError_t e = raise_smem(once, kern, T::kSmem);
  if (e != cudaSuccess) return e;
  Args a{};
  a.ps = l.ps;
  a.qs = l.qs;
  a.p_rows = l.p_rows;
  a.q_rows = l.q_rows;
  // rows and K may be just below 2^31: rounded up in 64 bits
  a.tiles_p = (int)((l.p_rows + 128ll * CG - 1) / (128 * CG));
  a.tiles_q = (int)((l.q_rows + (long long)NT - 1) / NT);
  const int slab = KIND == kBf16 ? 64 : 256;
  a.nk = (int)((l.k + (long long)slab - 1) / slab);
  a.sb = KIND == kBf16 ? 0 : l.k / (KIND == kNv ? 16 : 32);
  a.tma_scales = a.sb % 16 == 0;
  a.g0 = l.g0;
  a.g1 = l.g1;
  a.out = l.out;
  a.out_stride = l.out_stride;
  a.f32 = l.f32;
  a.wide = (reinterpret_cast<uintptr_t>(l.out) & 15) == 0 && l.out_stride % (l.f32 ? 4 : 8) == 0;
  a.status = l.status;
  const long long tiles = (long long)a.tiles_p * a.tiles_q;
  if (tiles > 0x3fffffff) return cudaErrorInvalidValue;
  a.split = split_for(tiles, (a.nk + T::kPer - 1) / T::kPer, CG, sms);
  const int team = CG * a.split;
  CUtensorMap pm, qm, psm{}, qsm{}, om{};
  const int elem = KIND == kBf16 ? 2 : 1;
  const long long width = KIND == kBf16 ? l.k : l.k / 2;
  e = make_map(&pm, l.p, elem, width, l.p_rows, l.p_stride, 128);
  if (e == cudaSuccess) e = make_map(&qm, l.q, elem, width, l.q_rows, l.q_stride, T::kQ);
  if (T::kBlocks && a.tma_scales) {
    if (e == cudaSuccess) e = make_scale_map(&psm, l.ps, a.sb, l.p_rows, 128);
    if (e == cudaSuccess) e = make_scale_map(&qsm, l.qs, a.sb, l.q_rows, NT);
  }
  if (e == cudaSuccess && !SWAP && a.wide && a.split == 1)
    e = make_out_map(&om, l.out, l.f32, l.q_rows, l.p_rows, l.out_stride * (l.f32 ? 4 : 2));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  const long long teams = tiles < sms / team ? tiles : sms / team;
  cfg.gridDim = dim3((unsigned)(teams * team));
  cfg.blockDim = dim3(T::kThreads);
  cfg.dynamicSmemBytes = T::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {(unsigned)team, 1, 1};
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, pm, qm, psm, qsm, om, a);
}

}  // namespace tg
}  // namespace moe

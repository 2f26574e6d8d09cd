// fp4_linear.cu -- the product of two 4-bit matrices on the tensor cores
// (formulas in moe_cache.h).
//
// tcgen05 block-scaled MMAs take both operands as packed e2m1 and multiply the
// block scales in: one MMA is 128 rows of P times NT rows of Q over 64 elements
// of K, products exact, sums in fp32 tensor memory.  P is the operand of 128
// rows.  With up to 64 tokens P are the weights and Q the tokens (SWAP; NT = 16,
// 32 or 64: weights stream from HBM once, and an MMA costs no more than its Q
// rows); with more, P are the tokens and Q the weights (NT = 64, 128 or 256).
//
// One CTA per SM works through tiles; warps:
//   0..3  epilogue: tensor memory -> registers -> global scales -> out;
//   4..7  block scales: rows of the scale banks to shared memory in the order
//         the MMA reads them, kAhead stages ahead in registers (16 bytes per row
//         and stage: TMA cannot interleave the rows' 4-byte words);
//   8     lane 0: TMA loads of the codes, one stage = 256 elements of K;
//   9     lane 0: MMAs; allocates the tensor memory.
// Scale order: the 32-bit word of row r and K step j lies at word (r / 32) of
// line r % 32 in a 512-byte block; a copy to tensor memory puts it in lane r % 32,
// column r / 32.  NVFP4: a word is the four scales of one 64-element step;
// MXFP4: the two scales of two steps, chosen by the instruction's scale ids.
// Where the tiles are fewer than half the SMs, S CTAs of a cluster share a tile:
// each sums its part of K and then, through distributed shared memory, its part
// of the tile's results over the ranks in ascending order.
// Every wait is bounded; on a timeout the CTA reports it, drains its copies and
// MMAs, frees its tensor memory and returns.
#include "block_ops.cuh"
#include "fp4.cuh"
#include "tc.cuh"

namespace moe {
namespace {

using namespace tc;

constexpr int kScaleWarp = 4, kTmaWarp = 8, kMmaWarp = 9;
constexpr int kThreads = 320;
constexpr int kAhead = 4;    // stages of scales in flight per thread
constexpr int kSlab = 256;   // K elements of a stage: 128 bytes of codes per row
constexpr int kMaxSplit = 8;

template <bool NV, int NT>
struct Shape {
  static constexpr int kQRows = NT < 128 ? 128 : NT;        // rows of the Q scale blocks
  static constexpr int kBlocks = NV ? 4 : 2;                // 32-bit scale words per row and stage
  static constexpr int kPScale = 128 * 4 * kBlocks;
  static constexpr int kQScale = kQRows * 4 * kBlocks;
  static constexpr int kStage = 128 * 128 + NT * 128 + kPScale + kQScale;
  static constexpr int kSmemMax = 226 * 1024;
  static constexpr int kFit = (kSmemMax - 1024 - 512) / kStage;
  static constexpr int kStages = kFit > 10 ? 10 : kFit;
  static constexpr int kAcc = NT <= 128 ? 2 : 1;            // accumulators
  static constexpr int kScaleCols = kBlocks * (4 + kQRows / 32);
  static constexpr int kScaleAt = kAcc * NT;                // first scale column
  static constexpr int kCols = kScaleAt + 2 * kScaleCols <= 128   ? 128
                               : kScaleAt + 2 * kScaleCols <= 256 ? 256
                                                                  : 512;
  static_assert(kScaleAt + 2 * kScaleCols <= 512 && kStage % 1024 == 0, "tile shape");
  static_assert(kStages * kStage >= 128 * (NT <= 128 ? NT : 0) * 4, "room for a partial tile");
};

struct Args {
  const uint8_t *ps, *qs;  // scale banks
  int p_rows, q_rows;
  int tiles_p, tiles_q;
  int nk;                  // stages of K
  int sb;                  // scale bytes per row
  int mode;                // 0: whole 16 (8) byte pieces, 1: words, 2: bytes
  int split;               // CTAs per tile
  const float *g0, *g1;
  void* out;
  long long out_stride;
  int f32, wide;           // wide: 32-byte stores fit the output's alignment
  unsigned long long* status;
};

template <int ST>
struct Ctl {
  uint64_t full[ST], scaled[ST], empty[ST];
  uint64_t acc_full[2], acc_empty[2], drain;
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

// the scale bytes of one row for stage ks, zero beyond the bank's row
template <bool NV>
__device__ __forceinline__ uint4 fetch_scales(const uint8_t* row, int ks, const Args& a) {
  uint4 v = make_uint4(0, 0, 0, 0);
  if (!row) return v;
  const int off = ks * (NV ? 16 : 8);
  if (a.mode == 0) {
    if (NV) return __ldg(reinterpret_cast<const uint4*>(row + off));
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(row + off));
    v.x = u.x;
    v.y = u.y;
    return v;
  }
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int i = 0; i < (NV ? 4 : 2); ++i) {
    if (a.mode == 1) {
      if (off + 4 * i < a.sb) w[i] = __ldg(reinterpret_cast<const uint32_t*>(row + off + 4 * i));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (off + 4 * i + j < a.sb) w[i] |= (uint32_t)__ldg(row + off + 4 * i + j) << (8 * j);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// row r's words into the blocks of a stage; `blocks` 512-byte blocks per word
template <bool NV>
__device__ __forceinline__ void put_scales(uint8_t* base, int r, int blocks, uint4 v) {
  uint8_t* p = base + (r >> 7) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4;
  *reinterpret_cast<uint32_t*>(p) = v.x;
  *reinterpret_cast<uint32_t*>(p + blocks * 512) = v.y;
  if (NV) {
    *reinterpret_cast<uint32_t*>(p + 2 * blocks * 512) = v.z;
    *reinterpret_cast<uint32_t*>(p + 3 * blocks * 512) = v.w;
  }
}

// Instruction descriptor: e2m1 x e2m1, K-major both, M 128, K 64, scales e4m3 or
// e8m0; `id` picks the scale bytes of a word.
template <bool NV>
__device__ __forceinline__ uint32_t idesc(int n, int id) {
  return ((uint32_t)id << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) |
         (NV ? 0u : 1u << 23) | ((128u >> 4) << 24) | ((uint32_t)id << 29);
}
template <bool NV>
__device__ __forceinline__ void mma(uint32_t d, uint64_t p, uint64_t q, uint32_t id, uint32_t sp,
                                    uint32_t sq, uint32_t acc) {
  if (NV)
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.scale_vec::4X [%0], %1, %2, %3, "
        "[%4], [%5], p;\n}\n" ::"r"(d),
        "l"(p), "l"(q), "r"(id), "r"(sp), "r"(sq), "r"(acc)
        : "memory");
  else
    asm volatile(
        "{\n .reg .pred p;\n setp.ne.b32 p, %6, 0;\n"
        " tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, "
        "[%4], [%5], p;\n}\n" ::"r"(d),
        "l"(p), "l"(q), "r"(id), "r"(sp), "r"(sq), "r"(acc)
        : "memory");
}

__device__ __forceinline__ void store_one(const Args& a, long long at, float v) {
  if (a.f32) static_cast<float*>(a.out)[at] = v;
  else static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(v);
}
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

template <bool NV, int NT, bool SWAP>
__global__ void __launch_bounds__(kThreads, 1)
linear_kernel(const __grid_constant__ CUtensorMap pmap, const __grid_constant__ CUtensorMap qmap,
              const Args a) {
  using T = Shape<NV, NT>;
  constexpr int ST = T::kStages;
  extern __shared__ uint8_t raw[];
  uint8_t* stg = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  __shared__ Ctl<ST> c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = blockIdx.x % a.split;
  const int k_lo = a.nk * rank / a.split, k_hi = a.nk * (rank + 1) / a.split, n_k = k_hi - k_lo;
  const int n_tiles = a.tiles_p * a.tiles_q, tile0 = blockIdx.x / a.split,
            step = gridDim.x / a.split;

  if (threadIdx.x == 0) {
    for (int i = 0; i < ST; ++i) {
      mbar_init(&c.full[i], 1);
      mbar_init(&c.scaled[i], 4);
      mbar_init(&c.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c.acc_full[i], 1);
      mbar_init(&c.acc_empty[i], 4);
    }
    mbar_init(&c.drain, 1);
    c.abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kMmaWarp) tmem_alloc(&c.tmem, T::kCols);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = c.tmem;

  if (warp == kTmaWarp) {
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int t = tile0; t < n_tiles && ok; t += step) {
        int tp, tq;
        tile_at(a, t, tp, tq);
        for (int ks = k_lo; ks < k_hi; ++ks, ++it) {
          const int s = it % ST;
          if (it >= ST && !wait_bar(&c.empty[s], (it / ST - 1) & 1, &c.abort_flag, a.status)) {
            ok = false;
            break;
          }
          uint8_t* p = stg + (size_t)s * T::kStage;
          mbar_expect(&c.full[s], 128 * 128 + NT * 128);
          tma_load(p, &pmap, ks * 128, tp * 128, &c.full[s]);
          tma_load(p + 128 * 128, &qmap, ks * 128, tq * NT, &c.full[s]);
        }
      }
      if (!ok)  // the copies in flight land before the CTA ends
        for (int i = it > ST ? it - ST : 0; i < it; ++i) drain_bar(&c.full[i % ST], (i / ST) & 1);
    }
    __syncwarp();
  } else if (warp == kMmaWarp) {
    if (lane == 0) {
      int it = 0, u = 0;
      bool ok = true;
      for (int t = tile0; t < n_tiles && ok; t += step, ++u) {
        const int b = u % T::kAcc;
        if (u >= T::kAcc &&
            !wait_bar(&c.acc_empty[b], (u / T::kAcc - 1) & 1, &c.abort_flag, a.status))
          break;
        fence_after();
        const uint32_t d = tmem + b * NT;
        for (int i = 0; i < n_k; ++i, ++it) {
          const int s = it % ST;
          if (!wait_bar(&c.full[s], (it / ST) & 1, &c.abort_flag, a.status) ||
              !wait_bar(&c.scaled[s], (it / ST) & 1, &c.abort_flag, a.status)) {
            ok = false;
            break;
          }
          fence_after();
          const uint32_t p0 = sa(stg + (size_t)s * T::kStage), q0 = p0 + 128 * 128;
          const uint32_t sp0 = q0 + NT * 128, sq0 = sp0 + T::kPScale;
          const uint32_t cp = tmem + T::kScaleAt + (it & 1) * T::kScaleCols, cq = cp + 4 * T::kBlocks;
          constexpr int QB = T::kQRows / 128;
#pragma unroll
          for (int j = 0; j < T::kBlocks; ++j) {
            copy_scales(cp + 4 * j, desc_scales(sp0 + 512 * j));
#pragma unroll
            for (int h = 0; h < QB; ++h)
              copy_scales(cq + 4 * (j * QB + h), desc_scales(sq0 + 512 * (j * QB + h)));
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int w = NV ? j : j / 2, id = NV ? 0 : 2 * (j & 1);
            mma<NV>(d, desc_tile(p0 + 32 * j), desc_tile(q0 + 32 * j), idesc<NV>(NT, id),
                    cp + 4 * w, cq + 4 * w * QB, (i | j) != 0);
          }
          mma_commit(&c.empty[s]);
        }
        if (!ok) break;
        mma_commit(&c.acc_full[b]);
      }
      if (it > 0) {  // every MMA has finished before the tensor memory is freed
        mma_commit(&c.drain);
        drain_bar(&c.drain, 0);
      }
    }
    __syncwarp();
  } else if (warp >= kScaleWarp) {
    const int r = threadIdx.x - 32 * kScaleWarp;  // 0 .. 127
    constexpr int QN = NT > 128 ? 2 : 1;          // Q rows per thread
    const int per_row = a.sb;
    // load cursor, kAhead stages in front of the stage being written
    int lt = tile0, lk = k_lo;
    const uint8_t *lp = nullptr, *lq[QN] = {};
    auto rows_of = [&](int t) {
      int tp, tq;
      tile_at(a, t, tp, tq);
      const long long p = (long long)tp * 128 + r;
      lp = p < a.p_rows ? a.ps + p * per_row : nullptr;
#pragma unroll
      for (int h = 0; h < QN; ++h) {
        const long long q = (long long)tq * NT + r + 128 * h;
        lq[h] = r < NT && q < a.q_rows ? a.qs + q * per_row : nullptr;
      }
    };
    uint4 vp[kAhead], vq[kAhead][QN];
    auto load = [&](int i) {
      if (lt >= n_tiles) return;
      vp[i] = fetch_scales<NV>(lp, lk, a);
#pragma unroll
      for (int h = 0; h < QN; ++h) vq[i][h] = fetch_scales<NV>(lq[h], lk, a);
      if (++lk == k_hi) {
        lk = k_lo;
        lt += step;
        if (lt < n_tiles) rows_of(lt);
      }
    };
    if (lt < n_tiles) rows_of(lt);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load(i);
    const int total = tile0 < n_tiles ? ((n_tiles - tile0 + step - 1) / step) * n_k : 0;
    bool ok = true;
    for (int it0 = 0; it0 < total && ok; it0 += kAhead) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int it = it0 + i, s = it % ST;
        if (it >= total || !ok) break;
        if (it >= ST) {
          bool w = true;
          if (lane == 0) w = wait_bar(&c.empty[s], (it / ST - 1) & 1, &c.abort_flag, a.status);
          ok = __shfl_sync(0xffffffffu, w, 0);
          if (!ok) break;
        }
        uint8_t* sp = stg + (size_t)s * T::kStage + 128 * 128 + NT * 128;
        put_scales<NV>(sp, r, 1, vp[i]);
        if (r < NT) {
#pragma unroll
          for (int h = 0; h < QN; ++h)
            put_scales<NV>(sp + T::kPScale, r + 128 * h, T::kQRows / 128, vq[i][h]);
        }
        load(i);
        fence_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&c.scaled[s]);
      }
    }
  } else {
    const float g = (a.g0 ? *a.g0 : 1.f) * (a.g1 ? *a.g1 : 1.f);
    int u = 0;
    for (int t = tile0; t < n_tiles; t += step, ++u) {
      const int b = u % T::kAcc;
      int tp, tq;
      tile_at(a, t, tp, tq);
      if (threadIdx.x == 0)
        c.epi_ok[u & 1] = wait_bar(&c.acc_full[b], (u / T::kAcc) & 1, &c.abort_flag, a.status);
      asm volatile("bar.sync 1, 128;" ::: "memory");
      if (!c.epi_ok[u & 1]) break;
      fence_after();
      const uint32_t acc = tmem + ((uint32_t)(32 * warp) << 16) + b * NT;
      const int pr = 32 * warp + lane;
      const long long p = (long long)tp * 128 + pr;
      constexpr int W = NT < 32 ? 16 : 32;  // columns read at a time
#pragma unroll 1
      for (int n0 = 0; n0 < NT; n0 += W) {
        const long long q0 = (long long)tq * NT + n0;
        if (q0 >= a.q_rows) break;
        uint32_t v[W];
        if constexpr (W == 16) tmem_ld16(acc + n0, v);
        else tmem_ld32(acc + n0, v);
        tmem_wait_ld();
        const int nq = (int)(a.q_rows - q0 < W ? a.q_rows - q0 : W);
        if (a.split > 1) {  // partial sums, [column][row], for the cluster's reduction
          float* part = reinterpret_cast<float*>(stg);
#pragma unroll
          for (int i = 0; i < W; ++i) part[(n0 + i) * 128 + pr] = __uint_as_float(v[i]);
        } else if (SWAP) {
          if (p < a.p_rows) {
#pragma unroll
            for (int i = 0; i < W; ++i)
              if (i < nq) store_one(a, (q0 + i) * a.out_stride + p, __uint_as_float(v[i]) * g);
          }
        } else if (p < a.p_rows) {
          const long long at = p * a.out_stride + q0;
          if (a.wide && nq == W) {
            if (a.f32) {
              float* o = static_cast<float*>(a.out) + at;
#pragma unroll
              for (int i = 0; i < W; i += 8) {
                uint32_t w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(__uint_as_float(v[i + j]) * g);
                store32(o + i, w);
              }
            } else {
              __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.out) + at;
#pragma unroll
              for (int i = 0; i < W; i += 16) {
                uint32_t w[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                  w[j] = pack2(__uint_as_float(v[i + 2 * j]) * g, __uint_as_float(v[i + 2 * j + 1]) * g);
                store32(o + i, w);
              }
            }
          } else {
#pragma unroll
            for (int i = 0; i < W; ++i)
              if (i < nq) store_one(a, at + i, __uint_as_float(v[i]) * g);
          }
        }
      }
      fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&c.acc_empty[b]);
    }
  }
  if (a.split > 1) {
    // one tile per cluster: rank's share of its results, summed over the ranks
    cluster_sync();
    int tp, tq;
    tile_at(a, tile0, tp, tq);
    const int cols = (int)(a.q_rows - (long long)tq * NT < NT ? a.q_rows - (long long)tq * NT : NT);
    const float g = (a.g0 ? *a.g0 : 1.f) * (a.g1 ? *a.g1 : 1.f);
    const uint32_t part = sa(stg);
    const int n = cols * 128;
    for (int i = rank * kThreads + threadIdx.x; i < n; i += a.split * kThreads) {
      // SWAP: neighbouring threads take neighbouring rows (outputs of one token);
      // else neighbouring columns
      const int col = SWAP ? i >> 7 : i % cols, row = SWAP ? i & 127 : i / cols;
      float v = 0.f;
      for (int k = 0; k < a.split; ++k) v += ld_peer(part + 4 * (col * 128 + row), k);
      const long long p = (long long)tp * 128 + row, q = (long long)tq * NT + col;
      if (p < a.p_rows && !c.abort_flag)
        store_one(a, SWAP ? q * a.out_stride + p : p * a.out_stride + q, v * g);
    }
    cluster_sync();  // a peer may still be reading this CTA's sums
  }
  fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    fence_after();
    tmem_free(tmem, T::kCols);
  }
}

template <bool NV, int NT, bool SWAP>
cudaError_t launch(const Fp4Linear& l, int sms, cudaStream_t s) {
  using T = Shape<NV, NT>;
  constexpr size_t kSmem = (size_t)T::kStages * T::kStage + 1024;
  auto kern = linear_kernel<NV, NT, SWAP>;
  static const cudaError_t set =
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (set != cudaSuccess) return set;
  Args a{};
  const uint8_t* pc = SWAP ? l.wc : l.xc;
  const uint8_t* qc = SWAP ? l.xc : l.wc;
  a.ps = SWAP ? l.ws : l.xs;
  a.qs = SWAP ? l.xs : l.ws;
  a.p_rows = SWAP ? l.n : l.rows;
  a.q_rows = SWAP ? l.rows : l.n;
  a.tiles_p = (a.p_rows + 127) / 128;
  a.tiles_q = (a.q_rows + NT - 1) / NT;
  a.nk = (l.k + kSlab - 1) / kSlab;
  a.sb = l.k / (NV ? 16 : 32);
  a.mode = a.sb % (NV ? 16 : 8) == 0 ? 0 : a.sb % 4 == 0 ? 1 : 2;
  a.g0 = l.xg;
  a.g1 = l.wg;
  a.out = l.out;
  a.out_stride = l.out_stride;
  a.f32 = l.f32;
  a.wide = (reinterpret_cast<uintptr_t>(l.out) & 31) == 0 && l.out_stride % (l.f32 ? 8 : 16) == 0;
  a.status = l.status;
  const long long tiles = (long long)a.tiles_p * a.tiles_q;
  if (tiles > 0x3fffffff) return cudaErrorInvalidValue;
  a.split = 1;
  if (NT <= 128)
    while (a.split < kMaxSplit && a.split * 2 <= a.nk && tiles * a.split * 2 <= sms) a.split *= 2;
  CUtensorMap pm, qm;
  cudaError_t e = make_map(&pm, pc, 1, l.k / 2, a.p_rows, l.k / 2, 128);
  if (e == cudaSuccess) e = make_map(&qm, qc, 1, l.k / 2, a.q_rows, l.k / 2, NT);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(a.split > 1 ? (unsigned)(tiles * a.split) : (unsigned)(tiles < sms ? tiles : sms));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {(unsigned)a.split, 1, 1};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, pm, qm, a);
}

template <bool NV>
cudaError_t by_rows(const Fp4Linear& l, int sms, cudaStream_t s) {
  if (l.rows <= 16) return launch<NV, 16, true>(l, sms, s);
  if (l.rows <= 32) return launch<NV, 32, true>(l, sms, s);
  if (l.rows <= 64) return launch<NV, 64, true>(l, sms, s);
  // the widest tile that still gives every SM one
  const long long tp = (l.rows + 127) / 128;
  if (tp * ((l.n + 255) / 256) >= sms) return launch<NV, 256, false>(l, sms, s);
  if (tp * ((l.n + 127) / 128) >= sms) return launch<NV, 128, false>(l, sms, s);
  return launch<NV, 64, false>(l, sms, s);
}

}  // namespace

cudaError_t launch_fp4_linear(const Fp4Linear& l, cudaStream_t s) {
  DeviceInfo d;
  const cudaError_t e = device_info(&d);
  if (e != cudaSuccess) return e;
  return l.nv ? by_rows<true>(l, d.sms, s) : by_rows<false>(l, d.sms, s);
}

}  // namespace moe

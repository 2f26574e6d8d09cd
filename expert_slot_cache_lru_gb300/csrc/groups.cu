// groups.cu -- a step's routes in order of their expert, and the routes' outputs back
// into their rows (formulas in moe_cache.h).
//
// The order is a stable counting sort in one launch of one cluster.  Every counting warp
// takes a run of consecutive routes: it counts them by expert in its own counters in
// shared memory (lanes with the same expert find one another by a ballot per bit of the id, the first
// adds for all, so no order of atomics matters; 65,536 routes of 256 experts 16.9 us, by
// __match_any_sync 21.5); prefixes over the warps, the cluster's CTAs (each CTA a slice of the
// experts) and the experts turn the counts into each warp's first places; and a second pass
// over the routes hands the places out.
//
// The combine is one pass bound by HBM: 16 bytes of a row per thread, the routes' loads
// in flight together.
#include "block_ops.cuh"
#include "linear.cuh"
#include "tc.cuh"

namespace moe {
namespace {

constexpr unsigned kAll = lin::kAll;
constexpr int kCtas = 16;  // of the largest cluster
// Routes up to which one CTA takes them, and up to which eight do (256 experts: 4,096 routes 9.9 us alone, 7.7 on
// eight, 8.6 on sixteen; 65,536 15.6 on eight, 12.3 on sixteen, whose scattered stores bound them).
constexpr int kAlone = 1024, kEight = 16384;

struct GroupArgs {
  const int32_t* ids;
  int32_t *offsets, *order, *pos;
  int routes, experts;
  int warps, per_warp;  // counting warps of a CTA, routes of a warp (a multiple of 32)
  int ctas, slice;      // experts of a CTA's slice
  int bits;             // of an id
};

// inclusive sum over the lanes
__device__ __forceinline__ unsigned warp_scan(unsigned v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned u = __shfl_up_sync(kAll, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// C: type of a warp's counters, which hold up to a CTA's routes; CTAS: a cluster's at most (one: all of it fits
// the block); PER: experts of the slice per thread at most
template <typename C, int THREADS, int CTAS, int PER>
__global__ void __launch_bounds__(THREADS, 1) group_kernel(const GroupArgs a) {
  extern __shared__ unsigned smem[];
  unsigned* first = smem;                              // [experts]: a CTA's routes, then its first place
  C* count = reinterpret_cast<C*>(smem + a.experts);   // [warps][experts]
  __shared__ unsigned sums[32], slice_total[CTAS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, E = a.experts;
  const int rank = CTAS == 1 ? 0 : (int)tc::cluster_rank();
  tc::pdl_trigger();
  for (int i = threadIdx.x; i < a.warps * E; i += THREADS) count[i] = 0;
  __syncthreads();
  tc::pdl_wait();
  const long long lo = ((long long)rank * a.warps + warp) * a.per_warp;
  const int n_mine = warp < a.warps ? (int)max(0ll, min((long long)a.per_warp, a.routes - lo)) : 0;
  C* mine = count + (warp < a.warps ? warp : 0) * E;
  const C* start = mine;

  // The place of each lane's route among those of its expert that the warp has seen, which are counted: lanes
  // with the same expert find one another by a ballot per bit, the first adds for all.
  auto count_in = [&](int e) {
    const unsigned valid = __ballot_sync(kAll, e >= 0);
    unsigned same = e >= 0 ? valid : 0u;
    for (int b = 0; b < a.bits; b += 4) {
#pragma unroll
      for (int z = 0; z < 4; ++z) {
        const bool on = e >> (b + z) & 1;
        const unsigned with = __ballot_sync(kAll, on);
        same &= on ? with : ~with;
      }
    }
    const unsigned below = __popc(same & ((1u << lane) - 1));
    unsigned rank = below;
    if (e >= 0) rank += mine[e];
    __syncwarp();
    if (e >= 0 && below == 0) mine[e] += (C)__popc(same);
    __syncwarp();
    return rank;
  };
  // routes, their experts (-1: none) and, in the first pass over a warp's only block, their ranks
  constexpr int U = 8;
  int id[U];
  unsigned rank_of[U];
  const bool once = a.per_warp <= 32 * U;  // all of a warp's routes at once: the ranks stay in registers
  auto load = [&](int i0) {
#pragma unroll
    for (int u = 0; u < U; ++u) id[u] = i0 + 32 * u + lane < n_mine ? a.ids[lo + i0 + 32 * u + lane] : -1;
#pragma unroll
    for (int u = 0; u < U; ++u) id[u] = (unsigned)id[u] < (unsigned)E ? id[u] : -1;
  };
  for (int i0 = 0; i0 < n_mine; i0 += 32 * U) {
    load(i0);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (i0 + 32 * u < n_mine) rank_of[u] = count_in(id[u]);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += THREADS) {  // counts to prefixes over the warps
    unsigned sum = 0;
    for (int w = 0; w < a.warps; ++w) {
      const unsigned c = count[w * E + e];
      count[w * E + e] = (C)sum;
      sum += c;
    }
    first[e] = sum;
  }
  if (CTAS > 1) tc::cluster_sync();
  else __syncthreads();
  // a thread's consecutive experts of the CTA's slice: routes of each CTA, and places within the slice
  const int per = (a.slice + THREADS - 1) / THREADS, e0 = rank * a.slice + threadIdx.x * per;
  const int e1 = min(min(e0 + per, (rank + 1) * a.slice), E);
  unsigned before[PER], sum = 0;  // before: an expert's routes and all before it of the thread's
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    before[j] = sum;
    if (j < per && e0 + j < e1) {
      if (CTAS == 1) {
        sum += first[e0 + j];
      } else {
        unsigned n[CTAS];
#pragma unroll
        for (int c = 0; c < CTAS; ++c)
          n[c] = c < a.ctas ? tc::load_at(tc::peer_addr(tc::sa(first + e0 + j), c)) : 0;
#pragma unroll
        for (int c = 0; c < CTAS; ++c) sum += n[c];
      }
    }
  }
  const unsigned incl = warp_scan(sum);
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  const unsigned in_warp = lane < THREADS / 32 ? sums[lane] : 0, upto = warp_scan(in_warp);
  const unsigned place = __shfl_sync(kAll, upto - in_warp, warp) + incl - sum;
  const unsigned total = __shfl_sync(kAll, upto, 31);  // of the slice
#pragma unroll
  for (int j = 0; j < PER; ++j)
    if (j < per && e0 + j < e1) {  // first place of the expert's routes in each CTA, within the slice
      unsigned at = place + before[j];
      if (CTAS == 1) {
        first[e0 + j] = at;
      } else {
        unsigned n[CTAS];
#pragma unroll
        for (int c = 0; c < CTAS; ++c)
          n[c] = c < a.ctas ? tc::load_at(tc::peer_addr(tc::sa(first + e0 + j), c)) : 0;
#pragma unroll
        for (int c = 0; c < CTAS; ++c) {
          if (c >= a.ctas) break;
          tc::store_at(tc::peer_addr(tc::sa(first + e0 + j), c), (int)at);
          at += n[c];
        }
      }
    }
  if (CTAS > 1) {
    if (threadIdx.x < a.ctas) tc::store_at(tc::peer_addr(tc::sa(slice_total + rank), threadIdx.x), (int)total);
    tc::cluster_sync();
  } else {
    if (threadIdx.x == 0) slice_total[0] = total;
    __syncthreads();
  }
  unsigned base[CTAS], all = 0;  // places before each slice
#pragma unroll
  for (int c = 0; c < CTAS; ++c) {
    base[c] = all;
    if (c < a.ctas) all += slice_total[c];
  }
  if (CTAS > 1) {
    for (int e = threadIdx.x; e < E; e += THREADS) {
      const int c = e / a.slice;
#pragma unroll
      for (int k = 1; k < CTAS; ++k)
        if (c == k) first[e] += base[k];
    }
  }
  unsigned mine_base = 0;
#pragma unroll
  for (int k = 1; k < CTAS; ++k)
    if (rank == k) mine_base = base[k];
#pragma unroll
  for (int j = 0; j < PER; ++j)
    if (j < per && e0 + j < e1) a.offsets[e0 + j] = (int32_t)(mine_base + place + before[j]);
  if (rank == 0 && threadIdx.x == 0) a.offsets[E] = (int32_t)all;
  __syncthreads();
  for (int i0 = 0; i0 < n_mine; i0 += 32 * U) {
    if (!once) {
      load(i0);
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (i0 + 32 * u < n_mine) rank_of[u] = count_in(id[u]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + 32 * u + lane;
      if (i >= n_mine) continue;
      const int e = id[u], r = (int)(lo + i);
      // counters hold the warp's first places and, in the second pass over a long run, its routes so far
      const int p = e < 0 ? -1 : (int)(first[e] + rank_of[u] + (once ? start[e] : 0));
      if (a.pos) a.pos[r] = p;
      if (a.order && p >= 0) a.order[p] = r;
    }
  }
  if (a.order)
    for (long long i = all + (long long)rank * THREADS + threadIdx.x; i < a.routes;
         i += (long long)a.ctas * THREADS)
      a.order[i] = -1;
}

template <typename C, int THREADS, int CTAS, int PER>
cudaError_t launch_group(const GroupArgs& a, int smem, cudaStream_t s) {
  auto kern = group_kernel<C, THREADS, CTAS, PER>;
  static tc::Once once, wide;
  cudaError_t e = tc::raise_smem(once, kern, 226 * 1024);
  if (e == cudaSuccess && CTAS > 8) e = tc::set_once(wide, kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(a.ctas);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim = {(unsigned)a.ctas, 1, 1};
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, a);
}

// V elements (8, or one) as they lie in memory, and their values
template <typename T, int V>
struct Raw {
  uint4 q[V * sizeof(T) / 16 > 0 ? V * sizeof(T) / 16 : 1];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (V == 1) {
      q[0].x = sizeof(T) == 4 ? *reinterpret_cast<const uint32_t*>(p) : *reinterpret_cast<const uint16_t*>(p) << 16;
    } else {
#pragma unroll
      for (int i = 0; i < (int)(V * sizeof(T) / 16); ++i) q[i] = reinterpret_cast<const uint4*>(p)[i];
    }
  }
  __device__ __forceinline__ float at(int i) const {
    const int per = 4 / sizeof(T) * 4;  // elements of 16 bytes
    const uint4& u = q[V == 1 ? 0 : i / per];
    const int word = V == 1 ? 0 : sizeof(T) == 4 ? i % 4 : i % 8 / 2;
    const uint32_t w = word == 0 ? u.x : word == 1 ? u.y : word == 2 ? u.z : u.w;
    if (V == 1 || sizeof(T) == 4) return __uint_as_float(w);
    return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
  }
};
template <int V>
__device__ __forceinline__ void store_v(float* p, const float (&v)[V]) {
  if constexpr (V == 1) {
    *p = v[0];
  } else {
#pragma unroll
    for (int i = 0; i < V; i += 4)
      *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  }
}
template <int V>
__device__ __forceinline__ void store_v(__nv_bfloat16* p, const float (&v)[V]) {
  if constexpr (V == 1) {
    *p = __float2bfloat16_rn(v[0]);
  } else {
    unsigned w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const unsigned*>(&b);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// Y, O: types of y and of add and out; V elements per thread.  A CTA takes `rows_per` rows at a time, or 256 of
// `pieces` pieces of one row; a thread loads U routes of its piece before it uses any, and the next piece's places and
// weights while it waits.
template <typename Y, typename O, int V, int U>
__global__ void __launch_bounds__(256) combine_kernel(const CombineArgs a, int pieces, int rows_per, int chunks) {
  tc::pdl_trigger();
  tc::pdl_wait();
  const int sub = rows_per > 1 ? threadIdx.x / pieces : 0, c0 = threadIdx.x - sub * pieces;
  const unsigned items = (unsigned)((a.rows + rows_per - 1ll) / rows_per * chunks);
  struct At {
    long long b, c;
    bool in;
  };
  auto at = [&](unsigned i) {
    const unsigned g = chunks > 1 ? i / chunks : i;
    const int piece = chunks > 1 ? (int)(i - g * chunks) * 256 + c0 : c0;
    const long long b = (long long)g * rows_per + sub;
    return At{b, (long long)piece * V, i < items && sub < rows_per && piece < pieces && b < a.rows};
  };
  int p[U], p_next[U];
  float f[U], f_next[U];
  auto places = [&](const At& x, int j0, int (&to)[U], float (&weight)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const bool in = x.in && j0 + u < a.k;
      to[u] = in ? a.pos[x.b * a.k + j0 + u] : -1;
      weight[u] = in ? a.w[x.b * a.k + j0 + u] : 0.f;
    }
  };
  unsigned i = blockIdx.x;
  places(at(i), 0, p, f);
  for (; i < items; i += gridDim.x) {
    const At x = at(i);
    float acc[V] = {};
    for (int j0 = 0; j0 < a.k; j0 += U) {
      Raw<Y, V> v[U];
      Raw<O, V> r;
#pragma unroll
      for (int u = 0; u < U; ++u)
        if ((unsigned)p[u] < (unsigned)a.y_rows) v[u].load(static_cast<const Y*>(a.y) + p[u] * a.y_stride + x.c);
      const bool add = j0 == 0 && a.add && x.in;
      if (add) r.load(static_cast<const O*>(a.add) + x.b * a.add_stride + x.c);
      if (j0 + U < a.k) places(x, j0 + U, p_next, f_next);
      else places(at(i + gridDim.x), 0, p_next, f_next);
      if (add)
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] = r.at(e);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if ((unsigned)p[u] < (unsigned)a.y_rows)
#pragma unroll
          for (int e = 0; e < V; ++e) acc[e] = fmaf(f[u], v[u].at(e), acc[e]);
        p[u] = p_next[u], f[u] = f_next[u];
      }
    }
    if (x.in) store_v<V>(static_cast<O*>(a.out) + x.b * a.out_stride + x.c, acc);
  }
}

template <typename Y, typename O, int V, int U>
cudaError_t launch_combine(const CombineArgs& a, cudaStream_t s) {
  tc::DeviceInfo d;
  cudaError_t e = tc::device_info(&d);
  if (e != cudaSuccess) return e;
  const int pieces = a.hidden / V, rows_per = pieces < 256 ? 256 / pieces : 1, chunks = (int)((pieces + 255ll) / 256);
  const long long items = (a.rows + rows_per - 1ll) / rows_per * chunks;
  if (items > 0x7fffffff) return cudaErrorInvalidValue;
  // as many CTAs as run at once (8,192 x 2 x 4,096 of two items a thread: 44 us with the three an SM that fit, 54 with
  // two, 55 with four; one item a thread is a little better: 43)
  static std::atomic<int> fit{0};
  int per_sm = fit.load(std::memory_order_relaxed);
  if (per_sm == 0) {
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, combine_kernel<Y, O, V, U>, 256, 0);
    if (e != cudaSuccess) return e;
    fit.store(per_sm, std::memory_order_relaxed);
  }
  const long long most = (long long)per_sm * d.sms;
  return tc::launch_early(combine_kernel<Y, O, V, U>, dim3((unsigned)(items < most ? items : most)), dim3(256), 0, s, a,
                          pieces, rows_per, chunks);
}
template <typename Y, typename O>
cudaError_t combine(const CombineArgs& a, cudaStream_t s) {
  auto whole = [](const void* p, long long stride, size_t e) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && stride * e % 16 == 0;
  };
  if (a.hidden % 8 == 0 && whole(a.y, a.y_stride, sizeof(Y)) &&
      whole(a.add, a.add ? a.add_stride : 0, sizeof(O)) && whole(a.out, a.out_stride, sizeof(O))) {
    if (a.k <= 2) return launch_combine<Y, O, 8, 2>(a, s);
    return launch_combine<Y, O, 8, 4>(a, s);  // of 8 routes too: 53.2 us for 8,192 x 8 x 2,048, eight at once 55.7
  }
  return launch_combine<Y, O, 1, 8>(a, s);
}

}  // namespace

cudaError_t launch_group_routes(const int32_t* ids, int routes, int experts, int32_t* offsets,
                                int32_t* order, int32_t* pos, cudaStream_t s) {
  GroupArgs a{ids, offsets, order, pos, routes, experts, 1, 32, 1, experts, 0};
  while ((experts - 1) >> a.bits) ++a.bits;
  // a CTA holds 32 warps of counters where they fit; of 16,384 experts 5 in 16 bits, 2 in 32
  const int room = 224 * 1024 - 4 * experts;
  auto plan = [&](int bytes) {
    const int most = room / (bytes * experts) < 32 ? room / (bytes * experts) : 32;
    a.ctas = routes <= kAlone ? 1 : routes <= kEight ? 8 : kCtas;
    a.slice = (experts + a.ctas - 1) / a.ctas;
    const long long runs = (routes + 31ll) / 32;  // 32 routes each
    a.warps = (int)(runs < most ? (runs > 0 ? runs : 1) : most);
    const long long all = (long long)a.warps * a.ctas;
    a.per_warp = (int)((runs + all - 1) / all * 32);
    if (a.per_warp == 0) a.per_warp = 32;
    return 4 * experts + a.warps * bytes * experts;
  };
  int smem = plan(2);
  const bool narrow = (long long)a.warps * a.per_warp <= 65535;
  if (!narrow) smem = plan(4);
  if (routes <= 256 && experts <= 1024) return launch_group<uint16_t, 256, 1, 4>(a, smem, s);
  if (a.ctas == 1) return launch_group<uint16_t, 1024, 1, 16>(a, smem, s);  // few routes: 16 bits hold them
  return narrow ? launch_group<uint16_t, 1024, kCtas, 2>(a, smem, s)
                : launch_group<uint32_t, 1024, kCtas, 2>(a, smem, s);
}

cudaError_t launch_combine(const CombineArgs& a, int y_dtype, int dtype, cudaStream_t s) {
  using B = __nv_bfloat16;
  if (dtype == MOE_T_BF16) return combine<B, B>(a, s);
  return y_dtype == MOE_T_BF16 ? combine<B, float>(a, s) : combine<float, float>(a, s);
}

}  // namespace moe

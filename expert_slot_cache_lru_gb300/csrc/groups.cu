// groups.cu -- a step's routes in order of their expert, and the routes' outputs back
// into their rows (formulas in moe_cache.h).
//
// The order is a stable counting sort in one launch of one cluster.  Every counting warp
// takes a run of consecutive routes: it counts them by expert in its own counters in
// shared memory (lanes with the same expert find one another, the first adds for all, so
// no order of atomics matters); prefixes over the warps, the cluster's CTAs and the experts
// turn the counts into each warp's first places; and a second pass over the routes hands
// the places out.
//
// The combine is one pass bound by HBM: 16 bytes of a row per thread, the routes' loads
// in flight together.
#include "block_ops.cuh"
#include "linear.cuh"
#include "tc.cuh"

namespace moe {
namespace {

constexpr unsigned kAll = lin::kAll;
constexpr int kMaxPer = 16;  // experts per thread of a block of 1,024

struct GroupArgs {
  const int32_t* ids;
  int32_t *offsets, *order, *pos;
  int routes, experts;
  int warps, per_warp;  // counting warps of a CTA, routes of a warp (a multiple of 32)
  int ctas;
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

// C: type of a warp's counters, which hold up to a CTA's routes
template <typename C, int THREADS>
__global__ void __launch_bounds__(THREADS, 1) group_kernel(const GroupArgs a) {
  extern __shared__ unsigned smem[];
  unsigned* first = smem;                              // [experts]: a CTA's routes, then its first place
  C* count = reinterpret_cast<C*>(smem + a.experts);   // [warps][experts]
  __shared__ unsigned sums[32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, E = a.experts;
  const int rank = a.ctas == 1 ? 0 : (int)tc::cluster_rank();
  tc::pdl_trigger();
  for (int i = threadIdx.x; i < a.warps * E; i += THREADS) count[i] = 0;
  __syncthreads();
  tc::pdl_wait();
  const long long lo = ((long long)rank * a.warps + warp) * a.per_warp;
  const int n_mine = warp < a.warps ? (int)max(0ll, min((long long)a.per_warp, a.routes - lo)) : 0;
  C* mine = count + (warp < a.warps ? warp : 0) * E;

  // the warp's routes, 32 at a time: f(route or -1, expert or -1, lanes with the same expert)
  auto each = [&](auto f) {
    int next = lane < n_mine ? a.ids[lo + lane] : -1;
    for (int i = 0; i < n_mine; i += 32) {
      const int id = next;
      if (i + 32 + lane < n_mine) next = a.ids[lo + i + 32 + lane];
      const int e = i + lane < n_mine && (unsigned)id < (unsigned)E ? id : -1;
      const unsigned same = __match_any_sync(kAll, e);
      f(i + lane < n_mine ? (int)(lo + i + lane) : -1, e, same);
      __syncwarp();
    }
  };
  each([&](int, int e, unsigned same) {
    if (e >= 0 && lane == __ffs(same) - 1) mine[e] += (C)__popc(same);
  });
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
  if (a.ctas > 1) tc::cluster_sync();
  else __syncthreads();
  // a thread's consecutive experts: routes of all CTAs, and of those before this one
  const int per = (E + THREADS - 1) / THREADS, e0 = threadIdx.x * per;
  unsigned all[kMaxPer], before[kMaxPer], sum = 0;
#pragma unroll
  for (int j = 0; j < kMaxPer; ++j) {
    all[j] = before[j] = 0;
    if (j < per && e0 + j < E) {
      for (int c = 0; c < a.ctas; ++c) {
        const unsigned n = a.ctas == 1 ? first[e0 + j] : tc::load_at(tc::peer_addr(tc::sa(first + e0 + j), c));
        all[j] += n;
        before[j] += c < rank ? n : 0;
      }
      sum += all[j];
    }
  }
  const unsigned incl = warp_scan(sum);
  if (lane == 31) sums[warp] = incl;
  if (a.ctas > 1) tc::cluster_sync();  // everyone has read the CTAs' counts
  else __syncthreads();
  const unsigned part = lane < THREADS / 32 ? sums[lane] : 0, upto = warp_scan(part);
  unsigned place = __shfl_sync(kAll, upto - part, warp) + incl - sum;
  const unsigned total = __shfl_sync(kAll, upto, 31);
#pragma unroll
  for (int j = 0; j < kMaxPer; ++j)
    if (j < per && e0 + j < E) {
      first[e0 + j] = place + before[j];
      if (rank == 0) a.offsets[e0 + j] = (int32_t)place;
      place += all[j];
    }
  if (rank == 0 && threadIdx.x == 0) a.offsets[E] = (int32_t)total;
  __syncthreads();
  each([&](int r, int e, unsigned same) {
    int p = -1;
    if (e >= 0) p = (int)(first[e] + mine[e] + __popc(same & ((1u << lane) - 1)));
    __syncwarp();
    if (e >= 0 && lane == __ffs(same) - 1) mine[e] += (C)__popc(same);
    if (r >= 0) {
      if (a.pos) a.pos[r] = p;
      if (a.order && p >= 0) a.order[p] = r;
    }
  });
  if (a.order)
    for (long long i = total + (long long)rank * THREADS + threadIdx.x; i < a.routes;
         i += (long long)a.ctas * THREADS)
      a.order[i] = -1;
}

template <typename C, int THREADS>
cudaError_t launch_group(const GroupArgs& a, int smem, cudaStream_t s) {
  auto kern = group_kernel<C, THREADS>;
  static tc::Once once;
  const cudaError_t e = tc::raise_smem(once, kern, 226 * 1024);
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

// Y, O: types of y and of add and out; V elements per thread, `pieces` per row
template <typename Y, typename O, int V>
__global__ void __launch_bounds__(256) combine_kernel(const CombineArgs a, int pieces) {
  tc::pdl_trigger();
  tc::pdl_wait();
  const long long i = (long long)blockIdx.x * 256 + threadIdx.x, b = i / pieces;
  if (b >= a.rows) return;
  const long long c = (i - b * pieces) * V;
  const Y* y = static_cast<const Y*>(a.y) + c;
  const int32_t* pos = a.pos + b * a.k;
  const float* w = a.w + b * a.k;
  float acc[V] = {};
  if (a.add) {
    Raw<O, V> r;
    r.load(static_cast<const O*>(a.add) + b * a.add_stride + c);
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] = r.at(e);
  }
  constexpr int U = sizeof(Y) == 4 ? 4 : 8;  // routes in flight: loaded before any is used
  for (int j0 = 0; j0 < a.k; j0 += U) {
    int p[U];
    float f[U];
    Raw<Y, V> v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      p[u] = j0 + u < a.k ? pos[j0 + u] : -1;
      f[u] = j0 + u < a.k ? w[j0 + u] : 0.f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if ((unsigned)p[u] < (unsigned)a.y_rows) v[u].load(y + p[u] * a.y_stride);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if ((unsigned)p[u] < (unsigned)a.y_rows)
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] = fmaf(f[u], v[u].at(e), acc[e]);
  }
  store_v<V>(static_cast<O*>(a.out) + b * a.out_stride + c, acc);
}

template <typename Y, typename O>
cudaError_t combine(const CombineArgs& a, cudaStream_t s) {
  auto whole = [](const void* p, long long stride, size_t e) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && stride * e % 16 == 0;
  };
  const bool wide = a.hidden % 8 == 0 && whole(a.y, a.y_stride, sizeof(Y)) &&
                    whole(a.add, a.add ? a.add_stride : 0, sizeof(O)) && whole(a.out, a.out_stride, sizeof(O));
  const int pieces = wide ? a.hidden / 8 : a.hidden;
  const long long blocks = ((long long)a.rows * pieces + 255) / 256;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)blocks), block(256);
  if (wide) return tc::launch_early(combine_kernel<Y, O, 8>, grid, block, 0, s, a, pieces);
  return tc::launch_early(combine_kernel<Y, O, 1>, grid, block, 0, s, a, pieces);
}

}  // namespace

cudaError_t launch_group_routes(const int32_t* ids, int routes, int experts, int32_t* offsets,
                                int32_t* order, int32_t* pos, cudaStream_t s) {
  GroupArgs a{ids, offsets, order, pos, routes, experts, 1, 32, 1};
  // a CTA holds 32 warps of counters where they fit, at least 3 (16,384 experts in 16 bits)
  const int room = 224 * 1024 - 4 * experts;
  auto plan = [&](int bytes) {
    const int most = room / (bytes * experts) < 32 ? room / (bytes * experts) : 32;
    a.ctas = routes <= 32 * 32 ? 1 : 8;
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
  const bool small = routes <= 256 && experts <= 1024;
  if (small) return launch_group<uint16_t, 256>(a, smem, s);
  return narrow ? launch_group<uint16_t, 1024>(a, smem, s) : launch_group<uint32_t, 1024>(a, smem, s);
}

cudaError_t launch_combine(const CombineArgs& a, int y_dtype, int dtype, cudaStream_t s) {
  using B = __nv_bfloat16;
  if (dtype == MOE_T_BF16) return combine<B, B>(a, s);
  return y_dtype == MOE_T_BF16 ? combine<B, float>(a, s) : combine<float, float>(a, s);
}

}  // namespace moe

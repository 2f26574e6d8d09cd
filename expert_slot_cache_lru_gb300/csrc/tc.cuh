// tc.cuh -- wrappers of the PTX that the tensor-core kernels of block_ops use:
// mbarriers with bounded waits, TMA tile loads, tensor memory, MMA issue.
#pragma once

#include <atomic>
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/moe_cache.h"

namespace moe {
namespace tc {

__device__ __forceinline__ uint32_t sa(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// ---------------------------------------------------------------- mbarriers
__device__ __forceinline__ void mbar_init(uint64_t* b, uint32_t n) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(sa(b)), "r"(n) : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(sa(b)) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint64_t* b, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(sa(b)), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ bool mbar_test(uint64_t* b, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(ok)
      : "r"(sa(b)), "r"(parity)
      : "memory");
  return ok != 0;
}

// A wait longer than this (about half a second) has failed: a whole product
// takes milliseconds.  Waits for copies and MMAs in flight keep that limit where
// the others are built with a shorter one, to see what follows a timeout.
constexpr long long kDrainCycles = 1000ll * 1000 * 1000;
#ifdef MOE_TC_WAIT_CYCLES
constexpr long long kWaitCycles = MOE_TC_WAIT_CYCLES;
#else
constexpr long long kWaitCycles = kDrainCycles;
#endif

__device__ __forceinline__ void raise_abort(int* flag, unsigned long long* status) {
  if (atomicExch(flag, 1) == 0 && status) atomicOr(status, (unsigned long long)MOE_STATUS_TIMEOUT);
}
// Bounded wait; false on timeout (which raises *flag) or when *flag is up.
__device__ __forceinline__ bool wait_bar(uint64_t* b, uint32_t parity, int* flag,
                                         unsigned long long* status) {
  if (mbar_test(b, parity)) return true;
  const long long t0 = clock64();
  while (!mbar_test(b, parity)) {
    if (*reinterpret_cast<volatile int*>(flag)) return false;
    if (clock64() - t0 > kWaitCycles) {
      raise_abort(flag, status);
      return false;
    }
  }
  return true;
}
// The same for a whole warp: one answer for all lanes.
__device__ __forceinline__ bool warp_wait(uint64_t* b, uint32_t parity, int* flag,
                                          unsigned long long* status) {
  return __all_sync(0xffffffffu, wait_bar(b, parity, flag, status));
}
// One lane of a converged warp.  The tensor-core and TMA instructions take warp-uniform
// operands: issued under this predicate by a warp that stays together they cost a
// few cycles, in a branch of lane 0 alone about 70 each.
__device__ __forceinline__ bool elect_one() {
  uint32_t yes;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n"
               : "=r"(yes));
  return yes != 0;
}
// Bounded wait that no flag ends, for copies and MMAs in flight; false on timeout.
__device__ __forceinline__ bool drain_bar(uint64_t* b, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_test(b, parity))
    if (clock64() - t0 > kDrainCycles) return false;
  return true;
}

// ---------------------------------------------------------------- TMA
// CG = 2: the copy of either CTA of a pair may signal a barrier of the pair's
// first CTA; `bar` is then a cluster address.
template <int CG>
__device__ __forceinline__ void tma_load(void* dst, const CUtensorMap* map, int x, int y,
                                         uint32_t bar) {
  if (CG == 1)
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], "
        "[%1, {%2, %3}], [%4];" ::"r"(sa(dst)),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];" ::"r"(sa(dst)),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// A tile from shared memory to the matrix of `map`, clipped at its edges; commit, and
// waits of the thread that issued it: until all but N copies have been read, or
// are done.
__device__ __forceinline__ void tma_store(const CUtensorMap* map, const void* src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(map),
               "r"(x), "r"(y), "r"(sa(src))
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void store_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void store_wait_done() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// ---------------------------------------------------------------- clusters
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t peer_addr(uint32_t saddr, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
  return a;
}
__device__ __forceinline__ void mbar_arrive_at(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
               : "memory");
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}
__device__ __forceinline__ void store_at(uint32_t cluster_addr, int v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(cluster_addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint32_t load_at(uint32_t cluster_addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(cluster_addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 lds4(uint32_t saddr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(saddr));
  return v;
}
// this thread's shared-memory writes, before the asynchronous copies that read them
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
// `bytes` (a multiple of 16) of this CTA's shared memory to a peer's, counted on
// the peer's barrier
__device__ __forceinline__ void copy_to_peer(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
      "r"(sa(src)), "r"(bytes), "r"(bar)
      : "memory");
}
// programmatic launch: let the next kernel of the stream start; wait for the
// previous one's results (for kernels started by launch_early)
__device__ __forceinline__ void pdl_trigger() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// ---------------------------------------------------------------- tcgen05
__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
template <int CG>
__device__ __forceinline__ void tmem_alloc(uint32_t* where, uint32_t cols) {
  if (CG == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sa(where)),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  } else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(sa(where)),
                 "r"(cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int CG>
__device__ __forceinline__ void tmem_free(uint32_t base, uint32_t cols) {
  if (CG == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols)
                 : "memory");
  else
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(base), "r"(cols)
                 : "memory");
}
// All MMAs issued so far, then one arrival at `bar`; CG = 2: at the barriers of
// the CTAs in `mask` at that offset.
template <int CG>
__device__ __forceinline__ void mma_commit(uint64_t* bar, uint16_t mask) {
  if (CG == 1)
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(sa(bar))
        : "memory");
  else
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
        "[%0], %1;" ::"r"(sa(bar)),
        "h"(mask)
        : "memory");
}
// Shared-memory descriptor of a K-major tile of 128-byte rows, 128-byte swizzle,
// 8-row groups 1,024 bytes apart.
__device__ __forceinline__ uint64_t desc_tile(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)1 << 16) |
         ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}

// Tensor memory, one warp: thread t holds lane (its quarter + t), column i in r[i].
#define MOE_TC_R8(r, o) \
  "r"(r[o]), "r"(r[o + 1]), "r"(r[o + 2]), "r"(r[o + 3]), "r"(r[o + 4]), "r"(r[o + 5]), "r"(r[o + 6]), "r"(r[o + 7])
#define MOE_TC_W8(r, o)                                                                        \
  "=r"(r[o]), "=r"(r[o + 1]), "=r"(r[o + 2]), "=r"(r[o + 3]), "=r"(r[o + 4]), "=r"(r[o + 5]), \
      "=r"(r[o + 6]), "=r"(r[o + 7])
template <int N>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&r)[N]) {
  static_assert(N == 16 || N == 32, "columns");
  if constexpr (N == 16)
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
        "%12, %13, %14, %15}, [%16];"
        : MOE_TC_W8(r, 0), MOE_TC_W8(r, 8)
        : "r"(taddr));
  else
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
        "%12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, "
        "%30, %31}, [%32];"
        : MOE_TC_W8(r, 0), MOE_TC_W8(r, 8), MOE_TC_W8(r, 16), MOE_TC_W8(r, 24)
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
// r into N columns from taddr, in pieces of 32, 16, 8 and 4
template <int N, int O = 0>
__device__ __forceinline__ void tmem_st_all(uint32_t taddr, const uint32_t (&r)[N]) {
  static_assert((N - O) % 4 == 0, "columns");
  if constexpr (N - O >= 32) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, "
        "%29, %30, %31};" ::MOE_TC_R8(r, O),
        MOE_TC_R8(r, O + 8), MOE_TC_R8(r, O + 16), MOE_TC_R8(r, O + 24), "r"(taddr + O)
        : "memory");
    tmem_st_all<N, O + 32>(taddr, r);
  } else if constexpr (N - O >= 16) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15};" ::MOE_TC_R8(r, O),
        MOE_TC_R8(r, O + 8), "r"(taddr + O)
        : "memory");
    tmem_st_all<N, O + 16>(taddr, r);
  } else if constexpr (N - O >= 8) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::MOE_TC_R8(r, O),
        "r"(taddr + O)
        : "memory");
    tmem_st_all<N, O + 8>(taddr, r);
  } else if constexpr (N - O == 4) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%4], {%0, %1, %2, %3};" ::"r"(r[O]),
                 "r"(r[O + 1]), "r"(r[O + 2]), "r"(r[O + 3]), "r"(taddr + O)
                 : "memory");
  }
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// ---------------------------------------------------------------- host side
// A 2-D map of rows of `row_bytes` (a multiple of 16; base 16-byte aligned) in
// tiles of 128 bytes x box_rows with the 128-byte swizzle; elements of elem
// bytes (1 or 2).  Outside the matrix a load reads zeros.
cudaError_t make_map(CUtensorMap* map, const void* base, int elem, long long width,
                     long long rows, long long row_bytes, int box_rows);
// The same for scale banks: tiles of 64 bytes, 64-byte swizzle.
cudaError_t make_scale_map(CUtensorMap* map, const void* base, long long row_bytes, long long rows,
                           int box_rows);

// Maps of `groups` matrices of bf16 rows, group_bytes apart, 128-byte swizzle: boxes of 64
// elements x 128 rows {k, n, groups}; gated, of 64 elements x 16 gate rows and their
// 16 up rows {k, 16, n / 16, 2, groups} (n a multiple of 16).
cudaError_t make_weight_map(CUtensorMap* map, const void* base, bool gated, long long k, long long n,
                            long long row_bytes, long long groups, long long group_bytes);

// A map of an output matrix of bf16 or fp32 in tiles of 32 x 32, 64- or 128-byte
// swizzle (rows a multiple of 16 bytes apart; base 16-byte aligned).
cudaError_t make_out_map(CUtensorMap* map, void* base, bool f32, long long width, long long rows,
                         long long row_bytes);

struct DeviceInfo {
  int sms;
};
// The current device's, read once per device.
cudaError_t device_info(DeviceInfo* out);

// Launches a kernel that may start while the one before it in the stream ends:
// it calls pdl_wait before it touches memory, and pdl_trigger first of all, for
// the next such kernel.  Hides launch and set-up, about a microsecond a call.
// Memory may still be written while such a kernel is already resident, so it reads with
// ordinary loads alone: non-coherent ones (__ldg, ld.global.nc, and what the compiler
// makes of const __restrict__ pointers) want data that stays as it is for a kernel's whole
// life, and may be moved above pdl_wait.
template <typename... P, typename... A>
cudaError_t launch_early(void (*kern)(P...), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                         const A&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, P(args)...);
}

// A kernel's attribute, set by its first launch on each device (devices past the 64th
// set it every time).
struct Once {
  std::atomic<unsigned long long> done{0};
};
template <typename K>
cudaError_t set_once(Once& once, K kern, cudaFuncAttribute attribute, int value) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
  if (once.done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, attribute, value);
  if (e == cudaSuccess) once.done.fetch_or(bit, std::memory_order_release);
  return e;
}
// Its dynamic shared-memory limit.
template <typename K>
cudaError_t raise_smem(Once& once, K kern, int bytes) {
  return set_once(once, kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

}  // namespace tc
}  // namespace moe

// block_norm.cu -- the seam between two blocks: post-norm, gate, residual add
// and the next block's pre-norm in one pass (formulas in moe_cache.h).
//
// One CTA per row; the row's h' stays in shared memory in fp32 between the two
// norms, so h and y are read once and h_out may be h itself.
#include "block_ops.cuh"

namespace moe {
namespace {

constexpr int kNormThreads = 256;

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void from_f(float v, float& o) { o = v; }
__device__ __forceinline__ void from_f(float v, __nv_bfloat16& o) { o = __float2bfloat16_rn(v); }

// sum over the CTA, the same bits in every thread
__device__ __forceinline__ float cta_sum(float v, float* red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.f;
  for (int i = 0; i < kNormThreads / 32; ++i) v += red[i];
  return v;
}

template <typename R>
__global__ void __launch_bounds__(kNormThreads) norm_kernel(NormArgs a) {
  extern __shared__ float row_h[];
  __shared__ float red[kNormThreads / 32];
  const int H = a.hidden;
  const long long b = blockIdx.x;
  const R* h = static_cast<const R*>(a.h) + b * a.h_stride;
  const __nv_bfloat16* y = a.y ? a.y + b * a.y_stride : nullptr;
  const __nv_bfloat16* gate = a.gate ? a.gate + b * a.gate_stride : nullptr;
  float inv = 1.f;
  if (a.post_w) {
    float s = 0.f;
    for (int i = threadIdx.x; i < H; i += kNormThreads) s += to_f(y[i]) * to_f(y[i]);
    inv = rsqrtf(cta_sum(s, red) / (float)H + a.eps);
  }
  float s = 0.f;
  for (int i = threadIdx.x; i < H; i += kNormThreads) {
    float v = to_f(h[i]);
    if (y) {
      float z = to_f(y[i]);
      if (a.post_w) z *= inv * (a.w_offset + to_f(a.post_w[i]));
      if (a.gate_kind == MOE_GATE_LINEAR) z *= to_f(gate[i]);
      if (a.gate_kind == MOE_GATE_SIGMOID) z /= 1.f + expf(-to_f(gate[i]));
      v += a.alpha * z;
    }
    row_h[i] = v;
    s += v * v;
    if (a.h_out) from_f(v, (static_cast<R*>(a.h_out) + b * a.ho_stride)[i]);
  }
  if (!a.pre_w) return;
  inv = rsqrtf(cta_sum(s, red) / (float)H + a.eps);
  for (int i = threadIdx.x; i < H; i += kNormThreads)
    from_f(row_h[i] * inv * (a.w_offset + to_f(a.pre_w[i])), a.x_out[b * a.xo_stride + i]);
}

template <typename R>
cudaError_t launch(const NormArgs& a, cudaStream_t s) {
  const size_t smem = sizeof(float) * (size_t)a.hidden;
  static const cudaError_t e = cudaFuncSetAttribute(
      norm_kernel<R>, cudaFuncAttributeMaxDynamicSharedMemorySize, 32768 * (int)sizeof(float));
  if (e != cudaSuccess) return e;
  norm_kernel<R><<<a.rows, kNormThreads, smem, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_block_norm(const NormArgs& a, int res_dtype, cudaStream_t s) {
  return res_dtype == MOE_T_F32 ? launch<float>(a, s) : launch<__nv_bfloat16>(a, s);
}

}  // namespace moe

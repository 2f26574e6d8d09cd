// block_ops.cuh -- the operators around the experts: argument records and the
// kernel launchers behind their C entry points (block_ops.cu).
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/moe_cache.h"

namespace moe {

// Stores e's text for moe_last_cuda_error; returns MOE_ERR_CUDA (moe_cache.cu).
int report_cuda(cudaError_t e, const char* what);

struct NormArgs {
  const void* h;
  const __nv_bfloat16 *y, *post_w, *gate, *pre_w;
  void* h_out;
  __nv_bfloat16* x_out;
  long long h_stride, y_stride, gate_stride, ho_stride, xo_stride;
  float alpha, w_offset, eps;
  int gate_kind, rows, hidden;
};
cudaError_t launch_block_norm(const NormArgs& a, int res_dtype, cudaStream_t s);

struct RouteArgs {
  const void* logits;  // [rows] stride
  long long stride;
  const float* bias;
  int32_t* ids;
  float* w;
  int rows, E, k, score, groups, topk_groups, group_top, renorm;
  float scale;
};
cudaError_t launch_route_select(const RouteArgs& a, int dtype, cudaStream_t s);
cudaError_t launch_route_logits(const __nv_bfloat16* x, long long x_stride,
                                const __nv_bfloat16* router, int rows, int hidden, int E, float* z,
                                unsigned long long* status, cudaStream_t s);

cudaError_t launch_fp4_quantize(bool nv, const void* src, int dtype, long long stride, int rows,
                                int cols, const float* g, uint8_t* codes, uint8_t* scales,
                                cudaStream_t s);
cudaError_t launch_fp4_dequantize(bool nv, const uint8_t* codes, const uint8_t* scales,
                                  const float* g, int rows, int cols, void* dst, int dtype,
                                  long long stride, cudaStream_t s);
cudaError_t launch_fp4_global_scale(const void* src, int dtype, long long stride, int rows,
                                    int cols, float* g, cudaStream_t s);

struct Fp4Linear {
  const uint8_t *xc, *xs, *wc, *ws;
  const float *xg, *wg;
  void* out;
  long long out_stride;
  int rows, n, k;
  bool nv, f32;
  unsigned long long* status;
};
cudaError_t launch_fp4_linear(const Fp4Linear& a, cudaStream_t s);

// A bf16 product, dense (offsets NULL: one group of all rows) or one per group.
struct Linear {
  const __nv_bfloat16 *x, *w, *bias;  // bias: [groups][n], or [groups][2 n]
  const void* res;
  void* out;
  long long x_stride, w_stride, group_stride, res_stride, out_stride;
  const int32_t *order, *offsets;
  int x_rows, per_row, groups;
  unsigned per_mul;  // r / per_row (launch_linear)
  int per_shift;
  int rows, n, k, act;
  bool gated, f32;
  float alpha;
  unsigned long long* status;
};
cudaError_t launch_linear(const Linear& a, cudaStream_t s);
// ... on the tensor cores: rows of whole 16-byte pieces, n a multiple of 16 if gated.
cudaError_t launch_linear_tc(const Linear& a, int sms, cudaStream_t s);

cudaError_t launch_group_routes(const int32_t* ids, int routes, int experts, int32_t* offsets,
                                int32_t* order, int32_t* pos, cudaStream_t s);

struct CombineArgs {
  const void *y, *add;
  void* out;
  const int32_t* pos;
  const float* w;
  long long y_stride, add_stride, out_stride;
  int y_rows, rows, k, hidden;
};
cudaError_t launch_combine(const CombineArgs& a, int y_dtype, int dtype, cudaStream_t s);

}  // namespace moe

// block_ops.cu -- host side of the operators around the experts: argument
// checks of their C entry points.  Everything is checked before anything is
// enqueued; nothing here allocates, waits or throws.
#include "block_ops.cuh"

namespace {

cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }
bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
size_t size_of(int dtype) { return dtype == MOE_T_F32 ? 4 : 2; }
bool is_dtype(int t) { return t == MOE_T_BF16 || t == MOE_T_F32; }

// A row stride in elements: 0 means `width`; false if rows would overlap.
bool take_stride(long long& stride, long long width) {
  if (stride == 0) stride = width;
  return stride >= width;
}

int done(cudaError_t e, const char* what) {
  return e == cudaSuccess ? MOE_OK : moe::report_cuda(e, what);
}

int check_choice(int n_rows, int E, int k, int score, int groups, int topk_groups, int group_top) {
  if (n_rows < 0 || E < 1 || k < 1 || k > E || groups < 1 || E % groups || topk_groups < 1 ||
      topk_groups > groups || (score != MOE_SCORE_SOFTMAX && score != MOE_SCORE_SIGMOID) ||
      (group_top != 1 && group_top != 2) || group_top > E / groups)
    return MOE_ERR_INVALID_ARG;
  if (E > 16384 || k > 32 || groups > 64) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// cols is a whole number of blocks
int check_banks(int wfmt, int rows, int cols, const float* g) {
  if (rows < 0 || cols < 1 || !aligned(g, 4)) return MOE_ERR_INVALID_ARG;
  if (wfmt == MOE_W_NVFP4) return cols % 16 ? MOE_ERR_INVALID_ARG : MOE_OK;
  if (wfmt == MOE_W_MXFP4) return cols % 32 || g ? MOE_ERR_INVALID_ARG : MOE_OK;
  return wfmt == MOE_W_BF16 || wfmt == MOE_W_Q4_0 ? MOE_ERR_UNSUPPORTED : MOE_ERR_INVALID_ARG;
}

// What the dense and the grouped product have in common; strides are filled in.
int check_linear(moe::Linear& l, int gated, int dtype) {
  if (l.rows < 0 || l.n < 1 || l.k < 1 || l.act < MOE_ACT_NONE || l.act > MOE_ACT_RELU ||
      (gated != 0 && gated != 1) || !is_dtype(dtype))
    return MOE_ERR_INVALID_ARG;
  l.gated = gated != 0;
  l.f32 = dtype == MOE_T_F32;
  const long long wide = l.gated ? 2ll * l.n : l.n;
  if (!take_stride(l.x_stride, l.k) || !take_stride(l.w_stride, l.k) ||
      !take_stride(l.out_stride, l.n) || !take_stride(l.res_stride, l.n))
    return MOE_ERR_INVALID_ARG;
  if (l.w_stride > (1ll << 62) / wide) return MOE_ERR_UNSUPPORTED;
  if (l.group_stride == 0) l.group_stride = wide * l.w_stride;
  if (l.group_stride < (wide - 1) * l.w_stride + l.k) return MOE_ERR_INVALID_ARG;
  if (l.rows == 0) return MOE_OK;
  const size_t e = size_of(dtype);
  if (!l.x || !l.w || !l.out || !aligned(l.x, 2) || !aligned(l.w, 2) || !aligned(l.bias, 2) ||
      !aligned(l.res, e) || !aligned(l.out, e) || !aligned(l.status, 8) ||
      (l.res == l.out && l.res_stride != l.out_stride) || l.out == l.x || l.out == l.w)
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

}  // namespace

extern "C" {

int moe_block_norm(const void* d_h, long long h_stride, const void* d_y, long long y_stride,
                   const void* d_post_w, const void* d_gate, long long gate_stride, int gate_kind,
                   float alpha, const void* d_pre_w, float w_offset, float eps, void* d_h_out,
                   long long h_out_stride, void* d_x_out, long long x_out_stride, int n_rows,
                   int hidden, int res_dtype, void* stream) {
  if (n_rows < 0 || hidden < 1 || !is_dtype(res_dtype) || gate_kind < MOE_GATE_NONE ||
      gate_kind > MOE_GATE_SIGMOID)
    return MOE_ERR_INVALID_ARG;
  if (hidden > 32768) return MOE_ERR_UNSUPPORTED;
  if ((gate_kind == MOE_GATE_NONE) != (d_gate == nullptr) || (!d_pre_w) != (!d_x_out) ||
      (!d_y && (d_post_w || d_gate)) || (!d_h_out && !d_x_out))
    return MOE_ERR_INVALID_ARG;
  if (!take_stride(h_stride, hidden) || !take_stride(y_stride, hidden) ||
      !take_stride(h_out_stride, hidden) || !take_stride(x_out_stride, hidden) ||
      (gate_stride != 0 && gate_stride < hidden))
    return MOE_ERR_INVALID_ARG;
  if (n_rows == 0) return MOE_OK;
  const size_t ra = size_of(res_dtype);
  if (!d_h || !aligned(d_h, ra) || !aligned(d_h_out, ra) || !aligned(d_y, 2) ||
      !aligned(d_post_w, 2) || !aligned(d_gate, 2) || !aligned(d_pre_w, 2) || !aligned(d_x_out, 2))
    return MOE_ERR_INVALID_ARG;
  if ((d_h_out == d_h && h_out_stride != h_stride) ||
      (d_x_out && d_x_out == d_y && x_out_stride != y_stride) || (d_x_out && d_x_out == d_h) ||
      (d_h_out && d_h_out == d_y) || (d_h_out && d_h_out == d_x_out))
    return MOE_ERR_INVALID_ARG;
  using B = __nv_bfloat16;
  moe::NormArgs a{};
  a.h = d_h;
  a.y = static_cast<const B*>(d_y);
  a.post_w = static_cast<const B*>(d_post_w);
  a.gate = static_cast<const B*>(d_gate);
  a.pre_w = static_cast<const B*>(d_pre_w);
  a.h_out = d_h_out;
  a.x_out = static_cast<B*>(d_x_out);
  a.h_stride = h_stride;
  a.y_stride = y_stride;
  a.gate_stride = gate_stride;
  a.ho_stride = h_out_stride;
  a.xo_stride = x_out_stride;
  a.alpha = alpha;
  a.w_offset = w_offset;
  a.eps = eps;
  a.gate_kind = gate_kind;
  a.rows = n_rows;
  a.hidden = hidden;
  return done(moe::launch_block_norm(a, res_dtype, as_stream(stream)), "moe_block_norm");
}

int moe_route(const void* d_x, long long x_stride, const void* d_router, const float* d_bias,
              int n_rows, int hidden, int n_experts, int k, int score, int n_groups,
              int topk_groups, int group_top, int renorm, float scale, float* d_logits,
              int32_t* d_ids, float* d_w, unsigned long long* d_status, void* stream) {
  const int rc = check_choice(n_rows, n_experts, k, score, n_groups, topk_groups, group_top);
  if (rc != MOE_OK) return rc;
  if (hidden < 1 || !take_stride(x_stride, hidden)) return MOE_ERR_INVALID_ARG;
  if (n_rows == 0) return MOE_OK;
  if (!d_x || !d_router || !d_logits || !d_ids || !d_w || !aligned(d_x, 2) ||
      !aligned(d_router, 2) || !aligned(d_bias, 4) || !aligned(d_logits, 4) ||
      !aligned(d_ids, 4) || !aligned(d_w, 4) || !aligned(d_status, 8))
    return MOE_ERR_INVALID_ARG;
  using B = __nv_bfloat16;
  const cudaError_t e =
      moe::launch_route_logits(static_cast<const B*>(d_x), x_stride, static_cast<const B*>(d_router),
                               n_rows, hidden, n_experts, d_logits, d_status, as_stream(stream));
  if (e != cudaSuccess) return done(e, "moe_route");
  const moe::RouteArgs a{d_logits, n_experts, d_bias,      d_ids,     d_w,    n_rows, n_experts, k,
                         score,    n_groups,  topk_groups, group_top, renorm, scale};
  return done(moe::launch_route_select(a, MOE_T_F32, as_stream(stream)), "moe_route");
}

int moe_route_logits(const void* d_logits, int dtype, long long logits_stride, const float* d_bias,
                     int n_rows, int n_experts, int k, int score, int n_groups, int topk_groups,
                     int group_top, int renorm, float scale, int32_t* d_ids, float* d_w,
                     void* stream) {
  const int rc = check_choice(n_rows, n_experts, k, score, n_groups, topk_groups, group_top);
  if (rc != MOE_OK) return rc;
  if (!is_dtype(dtype) || !take_stride(logits_stride, n_experts)) return MOE_ERR_INVALID_ARG;
  if (n_rows == 0) return MOE_OK;
  if (!d_logits || !d_ids || !d_w || !aligned(d_logits, size_of(dtype)) || !aligned(d_bias, 4) ||
      !aligned(d_ids, 4) || !aligned(d_w, 4))
    return MOE_ERR_INVALID_ARG;
  const moe::RouteArgs a{d_logits, logits_stride, d_bias,      d_ids,     d_w,    n_rows, n_experts,
                         k,        score,         n_groups, topk_groups, group_top, renorm, scale};
  return done(moe::launch_route_select(a, dtype, as_stream(stream)), "moe_route_logits");
}

int moe_fp4_quantize(int wfmt, const void* d_src, int dtype, long long src_stride, int rows,
                     int cols, const float* d_global, uint8_t* d_codes, uint8_t* d_scales,
                     void* stream) {
  const int rc = check_banks(wfmt, rows, cols, d_global);
  if (rc != MOE_OK) return rc;
  if (!is_dtype(dtype) || !take_stride(src_stride, cols)) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!d_src || !d_codes || !d_scales || !aligned(d_src, size_of(dtype)) || !aligned(d_codes, 16) ||
      !aligned(d_scales, 16))
    return MOE_ERR_INVALID_ARG;
  return done(moe::launch_fp4_quantize(wfmt == MOE_W_NVFP4, d_src, dtype, src_stride, rows, cols,
                                       d_global, d_codes, d_scales, as_stream(stream)),
              "moe_fp4_quantize");
}

int moe_fp4_dequantize(int wfmt, const uint8_t* d_codes, const uint8_t* d_scales,
                       const float* d_global, int rows, int cols, void* d_dst, int dtype,
                       long long dst_stride, void* stream) {
  const int rc = check_banks(wfmt, rows, cols, d_global);
  if (rc != MOE_OK) return rc;
  if (!is_dtype(dtype) || !take_stride(dst_stride, cols)) return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!d_dst || !d_codes || !d_scales || !aligned(d_dst, size_of(dtype)) || !aligned(d_codes, 16) ||
      !aligned(d_scales, 16))
    return MOE_ERR_INVALID_ARG;
  return done(moe::launch_fp4_dequantize(wfmt == MOE_W_NVFP4, d_codes, d_scales, d_global, rows,
                                         cols, d_dst, dtype, dst_stride, as_stream(stream)),
              "moe_fp4_dequantize");
}

int moe_fp4_global_scale(const void* d_src, int dtype, long long src_stride, int rows, int cols,
                         float* d_global, void* stream) {
  if (rows < 0 || cols < 1 || !is_dtype(dtype) || !take_stride(src_stride, cols))
    return MOE_ERR_INVALID_ARG;
  if (rows == 0) return MOE_OK;
  if (!d_src || !d_global || !aligned(d_src, size_of(dtype)) || !aligned(d_global, 4))
    return MOE_ERR_INVALID_ARG;
  return done(moe::launch_fp4_global_scale(d_src, dtype, src_stride, rows, cols, d_global,
                                           as_stream(stream)),
              "moe_fp4_global_scale");
}

int moe_fp4_linear(int wfmt, const uint8_t* d_x_codes, const uint8_t* d_x_scales,
                   const float* d_xg, const uint8_t* d_w_codes, const uint8_t* d_w_scales,
                   const float* d_wg, int n_rows, int n, int k, void* d_out, int dtype,
                   long long out_stride, unsigned long long* d_status, void* stream) {
  int rc = check_banks(wfmt, n_rows, k, d_xg);
  if (rc == MOE_OK) rc = check_banks(wfmt, n, k, d_wg);
  if (rc != MOE_OK) return rc;
  if (k % 32 || n < 1 || !is_dtype(dtype) || !take_stride(out_stride, n)) return MOE_ERR_INVALID_ARG;
  if (n_rows == 0) return MOE_OK;
  if (!d_x_codes || !d_x_scales || !d_w_codes || !d_w_scales || !d_out ||
      !aligned(d_x_codes, 16) || !aligned(d_x_scales, 16) || !aligned(d_w_codes, 16) ||
      !aligned(d_w_scales, 16) || !aligned(d_out, size_of(dtype)) || !aligned(d_status, 8))
    return MOE_ERR_INVALID_ARG;
  moe::Fp4Linear a{};
  a.xc = d_x_codes;
  a.xs = d_x_scales;
  a.wc = d_w_codes;
  a.ws = d_w_scales;
  a.xg = d_xg;
  a.wg = d_wg;
  a.out = d_out;
  a.out_stride = out_stride;
  a.rows = n_rows;
  a.n = n;
  a.k = k;
  a.nv = wfmt == MOE_W_NVFP4;
  a.f32 = dtype == MOE_T_F32;
  a.status = d_status;
  return done(moe::launch_fp4_linear(a, as_stream(stream)), "moe_fp4_linear");
}

int moe_linear(const void* d_x, long long x_stride, const void* d_w, long long w_stride,
               const void* d_bias, int act, int gated, const void* d_res, long long res_stride,
               float alpha, int n_rows, int n, int k, void* d_out, int dtype, long long out_stride,
               unsigned long long* d_status, void* stream) {
  using B = __nv_bfloat16;
  moe::Linear l{};
  l.x = static_cast<const B*>(d_x);
  l.w = static_cast<const B*>(d_w);
  l.bias = static_cast<const B*>(d_bias);
  l.res = d_res;
  l.out = d_out;
  l.x_stride = x_stride;
  l.w_stride = w_stride;
  l.res_stride = res_stride;
  l.out_stride = out_stride;
  l.x_rows = l.rows = n_rows;
  l.per_row = l.groups = 1;
  l.n = n;
  l.k = k;
  l.act = act;
  l.alpha = alpha;
  l.status = d_status;
  const int rc = check_linear(l, gated, dtype);
  if (rc != MOE_OK || n_rows == 0) return rc;
  return done(moe::launch_linear(l, as_stream(stream)), "moe_linear");
}

int moe_group_routes(const int32_t* d_ids, int n_routes, int n_experts, int32_t* d_offsets,
                     int32_t* d_order, int32_t* d_pos, void* stream) {
  if (n_routes < 0 || n_experts < 1) return MOE_ERR_INVALID_ARG;
  if (n_experts > 16384) return MOE_ERR_UNSUPPORTED;
  if (!d_offsets || (n_routes > 0 && !d_ids) || !aligned(d_ids, 4) || !aligned(d_offsets, 4) ||
      !aligned(d_order, 4) || !aligned(d_pos, 4) || d_offsets == d_ids || d_offsets == d_order ||
      d_offsets == d_pos || (d_order && (d_order == d_ids || d_order == d_pos)))
    return MOE_ERR_INVALID_ARG;
  return done(moe::launch_group_routes(d_ids, n_routes, n_experts, d_offsets, d_order, d_pos,
                                       as_stream(stream)),
              "moe_group_routes");
}

int moe_grouped_linear(const void* d_x, long long x_stride, int x_rows, const int32_t* d_order,
                       int per_row, const int32_t* d_offsets, int n_groups, const void* d_w,
                       long long w_group_stride, long long w_stride, const void* d_bias, int act,
                       int gated, int n_rows, int n, int k, void* d_out, int dtype,
                       long long out_stride, unsigned long long* d_status, void* stream) {
  using B = __nv_bfloat16;
  if (n_groups < 1 || per_row < 1 || x_rows < 0 || (!d_order && x_rows < n_rows))
    return MOE_ERR_INVALID_ARG;
  if (n_groups > 16384) return MOE_ERR_UNSUPPORTED;
  moe::Linear l{};
  l.x = static_cast<const B*>(d_x);
  l.w = static_cast<const B*>(d_w);
  l.bias = static_cast<const B*>(d_bias);
  l.out = d_out;
  l.x_stride = x_stride;
  l.w_stride = w_stride;
  l.group_stride = w_group_stride;
  l.out_stride = out_stride;
  l.order = d_order;
  l.offsets = d_offsets;
  l.x_rows = x_rows;
  l.per_row = per_row;
  l.groups = n_groups;
  l.rows = n_rows;
  l.n = n;
  l.k = k;
  l.act = act;
  l.alpha = 1.f;
  l.status = d_status;
  const int rc = check_linear(l, gated, dtype);
  if (rc != MOE_OK || n_rows == 0) return rc;
  if (!d_offsets || !aligned(d_offsets, 4) || !aligned(d_order, 4)) return MOE_ERR_INVALID_ARG;
  if (x_rows == 0) return MOE_OK;  // no place has a row
  return done(moe::launch_linear(l, as_stream(stream)), "moe_grouped_linear");
}

int moe_combine(const void* d_y, int y_dtype, long long y_stride, int y_rows, const int32_t* d_pos,
                const float* d_w, const void* d_add, long long add_stride, int n_rows, int k,
                int hidden, void* d_out, int dtype, long long out_stride, void* stream) {
  if (n_rows < 0 || y_rows < 0 || k < 1 || hidden < 1 || !is_dtype(y_dtype) || !is_dtype(dtype) ||
      (y_dtype == MOE_T_F32 && dtype != MOE_T_F32) || !take_stride(y_stride, hidden) ||
      !take_stride(add_stride, hidden) || !take_stride(out_stride, hidden))
    return MOE_ERR_INVALID_ARG;
  if (k > 1 << 30) return MOE_ERR_UNSUPPORTED;  // the kernel counts routes past the last in 32 bits
  if (n_rows == 0) return MOE_OK;
  const size_t e = size_of(dtype);
  if ((!d_y && y_rows > 0) || !d_pos || !d_w || !d_out || !aligned(d_y, size_of(y_dtype)) ||
      !aligned(d_pos, 4) || !aligned(d_w, 4) || !aligned(d_add, e) || !aligned(d_out, e) ||
      d_out == d_y || (d_out == d_add && out_stride != add_stride))
    return MOE_ERR_INVALID_ARG;
  moe::CombineArgs a{};
  a.y = d_y;
  a.add = d_add;
  a.out = d_out;
  a.pos = d_pos;
  a.w = d_w;
  a.y_stride = y_stride;
  a.add_stride = add_stride;
  a.out_stride = out_stride;
  a.y_rows = y_rows;
  a.rows = n_rows;
  a.k = k;
  a.hidden = hidden;
  return done(moe::launch_combine(a, y_dtype, dtype, as_stream(stream)), "moe_combine");
}

}  // extern "C"

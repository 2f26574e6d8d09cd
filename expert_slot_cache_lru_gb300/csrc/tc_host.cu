// tc_host.cu -- host helpers of the tensor-core kernels: TMA maps, device facts.
#include <atomic>

#include "tc.cuh"

namespace moe {
namespace tc {
namespace {

using Encode = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                            const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                            const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                            CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

Encode encoder() {
  static const Encode f = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<Encode>(p);
  }();
  return f;
}

}  // namespace

namespace {
cudaError_t encode(CUtensorMap* map, CUtensorMapDataType type, const void* base, long long width,
                   long long rows, long long row_bytes, int box_width, int box_rows,
                   CUtensorMapSwizzle swizzle) {
  const Encode f = encoder();
  if (!f) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {(cuuint64_t)width, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)row_bytes};
  const cuuint32_t box[2] = {(cuuint32_t)box_width, (cuuint32_t)box_rows};
  const cuuint32_t step[2] = {1, 1};
  const CUresult r = f(map, type, 2, const_cast<void*>(base), dims, strides, box, step,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                       CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}
}  // namespace

cudaError_t make_map(CUtensorMap* map, const void* base, int elem, long long width,
                     long long rows, long long row_bytes, int box_rows) {
  return encode(map, elem == 1 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base,
                width, rows, row_bytes, 128 / elem, box_rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

cudaError_t make_scale_map(CUtensorMap* map, const void* base, long long row_bytes, long long rows,
                           int box_rows) {
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, base, row_bytes, rows, row_bytes, 64, box_rows,
                CU_TENSOR_MAP_SWIZZLE_64B);
}

cudaError_t make_weight_map(CUtensorMap* map, const void* base, bool gated, long long k, long long n,
                            long long row_bytes, long long groups, long long group_bytes) {
  const Encode f = encoder();
  if (!f) return cudaErrorNotSupported;
  const cuuint64_t K = k, N = n, G = groups, rb = row_bytes, gb = group_bytes;
  const cuuint64_t dims3[3] = {K, N, G}, strides3[2] = {rb, gb};
  const cuuint64_t dims5[5] = {K, 16, N / 16, 2, G}, strides5[4] = {rb, 16 * rb, N * rb, gb};
  const cuuint32_t box3[3] = {64, 128, 1}, box5[5] = {64, 16, 1, 2, 1}, step[5] = {1, 1, 1, 1, 1};
  const CUresult r = f(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, gated ? 5 : 3, const_cast<void*>(base),
                       gated ? dims5 : dims3, gated ? strides5 : strides3, gated ? box5 : box3, step,
                       CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                       CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t make_out_map(CUtensorMap* map, void* base, bool f32, long long width, long long rows,
                         long long row_bytes) {
  return encode(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, base, width,
                rows, row_bytes, 32, 32, f32 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B);
}

cudaError_t device_info(DeviceInfo* out) {
  constexpr int kMax = 64;
  static std::atomic<int> sms[kMax];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int n = dev < kMax ? sms[dev].load(std::memory_order_relaxed) : 0;
  if (n == 0) {
    e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    if (dev < kMax) sms[dev].store(n, std::memory_order_relaxed);
  }
  out->sms = n;
  return cudaSuccess;
}

}  // namespace tc
}  // namespace moe

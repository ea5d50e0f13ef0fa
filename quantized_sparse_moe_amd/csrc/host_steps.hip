// C ABI of the steps around the experts' products: rows to buckets and back,
// SwiGLU, products with 4-bit weights. Host validation, then the launch.
// Nothing here allocates device memory, keeps state between calls or
// synchronises.
#include <hip/hip_runtime.h>

#include <climits>
#include <cstdint>

#include "qsmoe.h"
#include "kernels.hpp"

using namespace qsmoe;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

moe_status hip_status(hipError_t e) {
  return e == hipSuccess ? MOE_OK : e == hipErrorInvalidValue ? MOE_ERR_UNSUPPORTED : MOE_ERR_HIP;
}

bool is_dtype(int32_t d) { return d == MOE_DT_BF16 || d == MOE_DT_F32 || d == MOE_DT_F16; }
size_t size_of(int32_t d) { return d == MOE_DT_F32 ? 4 : 2; }

// The kernels index one row and all assignments with 32 bits.
constexpr int32_t kMaxSide = 1 << 20, kMaxRows = 1 << 30;

moe_status check_tokens(int32_t T, int32_t k, int32_t n, int32_t d) {
  if (T < 0 || k < 1 || n < 0 || d < 0) return MOE_ERR_INVALID_ARG;
  if (static_cast<int64_t>(T) * k > INT32_MAX) return MOE_ERR_INVALID_ARG;
  if (T * k > kMaxRows || n > kMaxRows || d > kMaxSide) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status check_swiglu(int64_t rows, int32_t inner) {
  if (rows < 0 || inner < 0) return MOE_ERR_INVALID_ARG;
  if (inner > kMaxSide || rows > INT64_MAX / 16 / kMaxSide) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status check_packed(int32_t dtype, int32_t out_dtype, int32_t format, int32_t group, int32_t T, int32_t k, int32_t N,
                      int32_t K, int32_t E) {
  if (T < 0 || k < 1 || N < 0 || K < 0 || E < 1 || !is_dtype(dtype) || !is_dtype(out_dtype)) return MOE_ERR_INVALID_ARG;
  if (static_cast<int64_t>(T) * k > INT32_MAX) return MOE_ERR_INVALID_ARG;
  if (E > 1024 || N > kMaxSide || K > kMaxSide || T * k > kMaxRows || dtype == MOE_DT_F32) return MOE_ERR_UNSUPPORTED;
  if (format == MOE_FMT_AFFINE ? group != 32 && group != 64 && group != 128 : format != MOE_FMT_MXFP4 || group != 32)
    return MOE_ERR_UNSUPPORTED;
  if (K < 1 || K % 32 != 0 || K % group != 0) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status check_packed_pointers(const void* x, const uint32_t* codes, const void* scales, const uint16_t* biases,
                               int32_t format, int32_t out_dtype, const void* out) {
  const bool affine = format == MOE_FMT_AFFINE;
  if (x == nullptr || codes == nullptr || scales == nullptr || out == nullptr || affine != (biases != nullptr))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, affine ? 2 : 1) || !aligned(biases, 2) ||
      !aligned(out, size_of(out_dtype)))
    return MOE_ERR_ALIGNMENT;
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_invert_perm(const int32_t* perm, int32_t n, int32_t size, int32_t* positions, int32_t* err,
                           hipStream_t stream) {
  if (n < 0 || size < 0) return MOE_ERR_INVALID_ARG;
  if (n > kMaxRows || size > kMaxRows) return MOE_ERR_UNSUPPORTED;
  if (size == 0) return MOE_OK;
  if (positions == nullptr || (n > 0 && perm == nullptr)) return MOE_ERR_INVALID_ARG;
  if (!aligned(perm, 4) || !aligned(positions, 4) || !aligned(err, 4)) return MOE_ERR_ALIGNMENT;
  return hip_status(launch_invert_perm(perm, n, size, positions, err, stream));
}

moe_status moe_gather_rows(const void* x, int32_t dtype, int32_t T, int32_t k, int32_t d, int32_t x_order,
                           const int32_t* perm, int32_t n, const float* topk_w, int32_t out_dtype, void* out,
                           int32_t* err, hipStream_t stream) {
  const moe_status s = check_tokens(T, k, n, d);
  if (s != MOE_OK) return s;
  if (!is_dtype(dtype) || !is_dtype(out_dtype) || (x_order != MOE_ROWS_TOKEN && x_order != MOE_ROWS_SLOT))
    return MOE_ERR_INVALID_ARG;
  if (n == 0 || d == 0) return MOE_OK;
  if (perm == nullptr || out == nullptr || (T > 0 && x == nullptr)) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, size_of(dtype)) || !aligned(out, size_of(out_dtype)) || !aligned(perm, 4) || !aligned(topk_w, 4) ||
      !aligned(err, 4))
    return MOE_ERR_ALIGNMENT;
  const GatherArgs g{x, perm, topk_w, out, err, dtype, out_dtype, T, k, n, d, x_order == MOE_ROWS_SLOT};
  return hip_status(launch_gather_rows(g, stream));
}

moe_status moe_combine_rows(const void* y, int32_t dtype, int32_t n, const int32_t* positions, const float* topk_w,
                            const void* y_shared, int32_t T, int32_t k, int32_t d, int32_t out_dtype, void* out,
                            int32_t* err, hipStream_t stream) {
  const moe_status s = check_tokens(T, k, n, d);
  if (s != MOE_OK) return s;
  if (!is_dtype(dtype) || !is_dtype(out_dtype) || (positions == nullptr && n != T * k)) return MOE_ERR_INVALID_ARG;
  if (T == 0 || d == 0) return MOE_OK;
  if (out == nullptr || (n > 0 && y == nullptr)) return MOE_ERR_INVALID_ARG;
  if (!aligned(y, size_of(dtype)) || !aligned(y_shared, size_of(dtype)) || !aligned(out, size_of(out_dtype)) ||
      !aligned(positions, 4) || !aligned(topk_w, 4) || !aligned(err, 4))
    return MOE_ERR_ALIGNMENT;
  const CombineArgs g{y, topk_w, positions, y_shared, out, err, dtype, out_dtype, T, k, n, d};
  return hip_status(launch_combine_rows(g, stream));
}

moe_status moe_combine_rows_grad(const void* dout, int32_t dout_dtype, const void* y, int32_t dtype, int32_t n,
                                 const int32_t* positions, const float* topk_w, int32_t T, int32_t k, int32_t d,
                                 void* dy, float* dw, int32_t* err, hipStream_t stream) {
  const moe_status s = check_tokens(T, k, n, d);
  if (s != MOE_OK) return s;
  if (!is_dtype(dtype) || !is_dtype(dout_dtype) || (positions == nullptr && n != T * k)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (topk_w == nullptr || dw == nullptr) return MOE_ERR_INVALID_ARG;
  if (d > 0 && (dout == nullptr || (n > 0 && (y == nullptr || dy == nullptr)))) return MOE_ERR_INVALID_ARG;
  if (!aligned(dout, size_of(dout_dtype)) || !aligned(y, size_of(dtype)) || !aligned(dy, size_of(dtype)) ||
      !aligned(positions, 4) || !aligned(topk_w, 4) || !aligned(dw, 4) || !aligned(err, 4))
    return MOE_ERR_ALIGNMENT;
  const CombineGradArgs g{dout, y, topk_w, positions, dy, dw, err, dtype, dout_dtype, T, k, n, d};
  return hip_status(launch_combine_rows_grad(g, stream));
}

moe_status moe_swiglu(const void* gu, int32_t dtype, int64_t rows, int32_t inner, void* h, hipStream_t stream) {
  const moe_status s = check_swiglu(rows, inner);
  if (s != MOE_OK) return s;
  if (!is_dtype(dtype)) return MOE_ERR_INVALID_ARG;
  if (rows == 0 || inner == 0) return MOE_OK;
  if (gu == nullptr || h == nullptr) return MOE_ERR_INVALID_ARG;
  if (!aligned(gu, size_of(dtype)) || !aligned(h, size_of(dtype))) return MOE_ERR_ALIGNMENT;
  return hip_status(launch_swiglu(gu, dtype, rows, inner, h, stream));
}

moe_status moe_swiglu_grad(const void* gu, int32_t dtype, const void* dh, int32_t dh_dtype, int64_t rows,
                           int32_t inner, void* dgu, hipStream_t stream) {
  const moe_status s = check_swiglu(rows, inner);
  if (s != MOE_OK) return s;
  if (!is_dtype(dtype) || !is_dtype(dh_dtype)) return MOE_ERR_INVALID_ARG;
  if (rows == 0 || inner == 0) return MOE_OK;
  if (gu == nullptr || dh == nullptr || dgu == nullptr) return MOE_ERR_INVALID_ARG;
  if (!aligned(gu, size_of(dtype)) || !aligned(dh, size_of(dh_dtype)) || !aligned(dgu, size_of(dtype)))
    return MOE_ERR_ALIGNMENT;
  return hip_status(launch_swiglu_grad(gu, dtype, dh, dh_dtype, rows, inner, dgu, stream));
}

moe_status moe_matmul_packed(const void* x, int32_t dtype, const uint32_t* codes, const void* scales,
                           const uint16_t* biases, int32_t format, int32_t group, int32_t M, int32_t N, int32_t K,
                           int32_t out_dtype, void* out, hipStream_t stream) {
  moe_status s = check_packed(dtype, out_dtype, format, group, M, 1, N, K, 1);
  if (s != MOE_OK) return s;
  if (M == 0 || N == 0) return MOE_OK;
  if ((s = check_packed_pointers(x, codes, scales, biases, format, out_dtype, out)) != MOE_OK) return s;
  const PackedArgs p{x, codes, scales, biases, dtype, out_dtype, M, 1, 1, N, K, group, nullptr, nullptr,
                       MOE_ROWS_BUCKET, MOE_ROWS_BUCKET, out, nullptr};
  return hip_status(launch_product_packed(p, stream));
}

moe_status moe_grouped_matmul_packed(const void* x, int32_t dtype, const uint32_t* codes, const void* scales,
                                   const uint16_t* biases, int32_t format, int32_t group, int32_t T, int32_t k,
                                   int32_t N, int32_t K, int32_t E, const int32_t* offsets, const int32_t* perm,
                                   int32_t x_order, int32_t out_order, int32_t out_dtype, void* out, int32_t* err,
                                   hipStream_t stream) {
  moe_status s = check_packed(dtype, out_dtype, format, group, T, k, N, K, E);
  if (s != MOE_OK) return s;
  if (x_order != MOE_ROWS_BUCKET && x_order != MOE_ROWS_TOKEN && x_order != MOE_ROWS_SLOT) return MOE_ERR_INVALID_ARG;
  if (out_order != MOE_ROWS_BUCKET && out_order != MOE_ROWS_SLOT) return MOE_ERR_INVALID_ARG;
  if (T == 0 || N == 0) return MOE_OK;
  if (offsets == nullptr || ((x_order != MOE_ROWS_BUCKET || out_order != MOE_ROWS_BUCKET) && perm == nullptr))
    return MOE_ERR_INVALID_ARG;
  if ((s = check_packed_pointers(x, codes, scales, biases, format, out_dtype, out)) != MOE_OK) return s;
  if (!aligned(offsets, 4) || !aligned(perm, 4) || !aligned(err, 4)) return MOE_ERR_ALIGNMENT;
  const PackedArgs p{x, codes, scales, biases, dtype, out_dtype, T, k, E, N, K, group, offsets, perm, x_order,
                       out_order, out, err};
  return hip_status(launch_product_packed(p, stream));
}

}  // extern "C"

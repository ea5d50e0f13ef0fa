// C ABI of the block-scaled FP8 quantisers and the products grouped by
// expert: host validation, then one launch. Nothing here allocates device
// memory, keeps state between calls or synchronises.
#include <hip/hip_runtime.h>

#include <climits>
#include <cstdint>

#include "qsmoe.h"
#include "kernels.hpp"

using namespace qsmoe;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

moe_status hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

bool is_dtype(int32_t d) { return d == MOE_DT_BF16 || d == MOE_DT_F32 || d == MOE_DT_F16; }

// out_dtype of the FP8 products: its flag and the type itself.
int32_t take_f32_sums(int32_t* out_dtype) {
  const int32_t flag = *out_dtype & MOE_SUMS_F32;
  *out_dtype &= ~MOE_SUMS_F32;
  return flag != 0;
}

// The kernels index one expert's tiles and all positions, rounded up to a
// tile, with 32 bits.
constexpr int32_t kMaxSide = 1 << 20, kMaxRows = 1 << 30;

moe_status check_groups(int32_t T, int32_t k, int32_t N, int32_t K, int32_t E) {
  if (T < 0 || k < 1 || N < 0 || K < 0 || E < 1) return MOE_ERR_INVALID_ARG;
  if (static_cast<int64_t>(T) * k > INT32_MAX) return MOE_ERR_INVALID_ARG;
  if (E > 1024 || N > kMaxSide || K > kMaxSide || T * k > kMaxRows) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

moe_status check_orders(int32_t in, int32_t out, bool in_token_ok, const int32_t* perm) {
  if (in != MOE_ROWS_BUCKET && in != MOE_ROWS_SLOT && !(in_token_ok && in == MOE_ROWS_TOKEN))
    return MOE_ERR_INVALID_ARG;
  if (out != MOE_ROWS_BUCKET && out != MOE_ROWS_SLOT) return MOE_ERR_INVALID_ARG;
  if ((in != MOE_ROWS_BUCKET || out != MOE_ROWS_BUCKET) && perm == nullptr) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_quantize_block(const void* x, int32_t dtype, int64_t matrices, int64_t rows, int32_t cols,
                              int32_t block_rows, int32_t pow2, uint8_t* codes, float* scales, int32_t* err,
                              hipStream_t stream) {
  if (matrices < 0 || rows < 0 || cols < 0 || !is_dtype(dtype)) return MOE_ERR_INVALID_ARG;
  if ((block_rows != 1 && block_rows != 128) || cols % 16 != 0) return MOE_ERR_UNSUPPORTED;
  if (matrices == 0 || rows == 0 || cols == 0) return MOE_OK;
  if (matrices > INT64_MAX / rows || matrices * rows > (INT64_MAX / 4) / cols) return MOE_ERR_UNSUPPORTED;
  if (x == nullptr || codes == nullptr || scales == nullptr) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 4) || !aligned(err, 4)) return MOE_ERR_ALIGNMENT;
  const hipError_t e = launch_quantize_block(x, dtype, matrices, rows, cols, block_rows, pow2 != 0, codes, scales,
                                             err, stream);
  return e == hipErrorInvalidValue ? MOE_ERR_UNSUPPORTED : hip_status(e);
}

moe_status moe_swiglu_quantize_block(const void* gu, int32_t dtype, int64_t rows, int32_t inner, int32_t pow2,
                                     uint8_t* codes, float* scales, int32_t* err, hipStream_t stream) {
  if (rows < 0 || inner < 0 || !is_dtype(dtype)) return MOE_ERR_INVALID_ARG;
  if (inner % 16 != 0 || inner > INT32_MAX / 2) return MOE_ERR_UNSUPPORTED;
  if (rows == 0 || inner == 0) return MOE_OK;
  if (rows > (INT64_MAX / 8) / inner) return MOE_ERR_UNSUPPORTED;
  if (gu == nullptr || codes == nullptr || scales == nullptr) return MOE_ERR_INVALID_ARG;
  if (!aligned(gu, 16) || !aligned(codes, 16) || !aligned(scales, 4) || !aligned(err, 4)) return MOE_ERR_ALIGNMENT;
  const hipError_t e = launch_swiglu_quantize_block(gu, dtype, rows, inner, pow2 != 0, codes, scales, err, stream);
  return e == hipErrorInvalidValue ? MOE_ERR_UNSUPPORTED : hip_status(e);
}

moe_status moe_matmul_block(const uint8_t* a, const float* a_scales, const uint8_t* b, const float* b_scales,
                            int32_t M, int32_t N, int32_t K, int32_t out_dtype, void* out, hipStream_t stream) {
  moe_status s = check_groups(M, 1, N, K, 1);
  if (s != MOE_OK) return s;
  const int32_t f32_sums = take_f32_sums(&out_dtype);
  if (!is_dtype(out_dtype)) return MOE_ERR_INVALID_ARG;
  if (K % 16 != 0 || N % 8 != 0) return MOE_ERR_UNSUPPORTED;
  if (M == 0 || N == 0) return MOE_OK;
  if (out == nullptr || (K > 0 && (a == nullptr || a_scales == nullptr || b == nullptr || b_scales == nullptr)))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(a, 16) || !aligned(b, 16) || !aligned(out, 16) || !aligned(a_scales, 4) || !aligned(b_scales, 4))
    return MOE_ERR_ALIGNMENT;
  ProductArgs p{a, a_scales, b, b_scales, kTypeE4m3, out_dtype, M, 1, 1, N, K, 0, f32_sums, nullptr, nullptr,
                MOE_ROWS_BUCKET, MOE_ROWS_BUCKET, out, nullptr};
  const hipError_t e = launch_product(p, stream);
  return e == hipErrorInvalidValue ? MOE_ERR_UNSUPPORTED : hip_status(e);
}

moe_status moe_grouped_matmul_block(const uint8_t* a, const float* a_scales, const uint8_t* w, const float* w_scales,
                                    int32_t T, int32_t k, int32_t N, int32_t K, int32_t E, const int32_t* offsets,
                                    const int32_t* perm, int32_t a_order, int32_t out_order, int32_t out_dtype,
                                    void* out, int32_t* err, hipStream_t stream) {
  moe_status s = check_groups(T, k, N, K, E);
  if (s != MOE_OK) return s;
  const int32_t f32_sums = take_f32_sums(&out_dtype);
  if (!is_dtype(out_dtype)) return MOE_ERR_INVALID_ARG;
  if (K % 16 != 0 || N % 8 != 0) return MOE_ERR_UNSUPPORTED;
  if ((s = check_orders(a_order, out_order, true, T > 0 ? perm : reinterpret_cast<const int32_t*>(4))) != MOE_OK)
    return s;
  if (T == 0 || N == 0) return MOE_OK;
  if (offsets == nullptr || out == nullptr) return MOE_ERR_INVALID_ARG;
  if (K > 0 && (a == nullptr || a_scales == nullptr || w == nullptr || w_scales == nullptr))
    return MOE_ERR_INVALID_ARG;
  if (!aligned(a, 16) || !aligned(w, 16) || !aligned(out, 16) || !aligned(a_scales, 4) || !aligned(w_scales, 4) ||
      !aligned(offsets, 4) || !aligned(perm, 4) || !aligned(err, 4))
    return MOE_ERR_ALIGNMENT;
  ProductArgs p{a, a_scales, w, w_scales, kTypeE4m3, out_dtype, T, k, E, N, K, 0, f32_sums, offsets, perm, a_order,
                out_order, out, err};
  const hipError_t e = launch_product(p, stream);
  return e == hipErrorInvalidValue ? MOE_ERR_UNSUPPORTED : hip_status(e);
}

moe_status moe_grouped_matmul(const void* x, const void* w, int32_t dtype, int32_t T, int32_t k, int32_t N, int32_t K,
                              int32_t E, const int32_t* offsets, const int32_t* perm, int32_t x_order,
                              int32_t out_order, int32_t transposed, int32_t out_dtype, void* out, int32_t* err,
                              hipStream_t stream) {
  moe_status s = check_groups(T, k, N, K, E);
  if (s != MOE_OK) return s;
  if (!is_dtype(out_dtype) || !is_dtype(dtype)) return MOE_ERR_INVALID_ARG;
  if (dtype == MOE_DT_F32 || K % 8 != 0 || N % 8 != 0) return MOE_ERR_UNSUPPORTED;
  if ((s = check_orders(x_order, out_order, true, T > 0 ? perm : reinterpret_cast<const int32_t*>(4))) != MOE_OK)
    return s;
  const int32_t C = transposed ? K : N, Q = transposed ? N : K;
  if (T == 0 || C == 0) return MOE_OK;
  if (offsets == nullptr || out == nullptr || (Q > 0 && (x == nullptr || w == nullptr))) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(out, 16) || !aligned(offsets, 4) || !aligned(perm, 4) ||
      !aligned(err, 4))
    return MOE_ERR_ALIGNMENT;
  ProductArgs p{x, nullptr, w, nullptr, dtype, out_dtype, T, k, E, C, Q, transposed != 0, 0, offsets, perm, x_order,
                out_order, out, err};
  const hipError_t e = launch_product(p, stream);
  return e == hipErrorInvalidValue ? MOE_ERR_UNSUPPORTED : hip_status(e);
}

moe_status moe_grouped_matmul_dw(const void* x, const void* dy, int32_t dtype, int32_t T, int32_t k, int32_t N,
                                 int32_t K, int32_t E, const int32_t* offsets, const int32_t* perm, int32_t x_order,
                                 int32_t dy_order, int32_t out_dtype, void* out, int32_t* err, hipStream_t stream) {
  moe_status s = check_groups(T, k, N, K, E);
  if (s != MOE_OK) return s;
  if (!is_dtype(out_dtype) || !is_dtype(dtype)) return MOE_ERR_INVALID_ARG;
  if (dtype == MOE_DT_F32 || K % 8 != 0 || N % 8 != 0) return MOE_ERR_UNSUPPORTED;
  if ((s = check_orders(x_order, dy_order, true, T > 0 ? perm : reinterpret_cast<const int32_t*>(4))) != MOE_OK)
    return s;
  if (N == 0 || K == 0) return MOE_OK;
  if (out == nullptr || (T > 0 && (offsets == nullptr || x == nullptr || dy == nullptr))) return MOE_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(dy, 16) || !aligned(out, 16) || !aligned(offsets, 4) || !aligned(perm, 4) ||
      !aligned(err, 4))
    return MOE_ERR_ALIGNMENT;
  DwArgs p{x, dy, dtype, out_dtype, T, k, E, N, K, offsets, perm, x_order, dy_order, out, err};
  const hipError_t e = launch_product_dw(p, stream);
  return e == hipErrorInvalidValue ? MOE_ERR_UNSUPPORTED : hip_status(e);
}

}  // extern "C"

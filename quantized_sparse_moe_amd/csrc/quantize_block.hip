// Block-scaled FP8 quantisation: E4M3 codes with one fp32 scale per block of
// 128 columns and 1 row (activations) or 128 rows (weights), and the SwiGLU
// between an expert's two products fused in front of the 1 x 128 form.
// Per block, every step in fp32 with IEEE rounding:
//   s = max(amax / 448, 2^-126), raised to a power of two first if asked,
//   code = e4m3_rne(x * (1 / s)).
// A block with a NaN or an infinity gets the scale NaN and codes 0.
//
// Both kernels read each element once and hold it in registers between the
// maximum and the conversion, 16 elements per lane, so that a lane's codes
// leave as one 16-byte store; memory bounds them. 32 x [2048][4096] bf16
// weights in 128 x 128 blocks: 149 us, 5.4 TB/s (a large copy: 4.9). The
// SwiGLU divides by way of a reciprocal: 24576 rows of 2048 45 us, 5.7 TB/s;
// with the division itself the VALU bounds it at 55 us. One row of 4096: 7.2
// us a call, the host's side of it.
#include "common.hpp"
#include "kernels.hpp"

namespace qsmoe {

namespace {

// Blocks of 128 in a row; cols + 127 may pass 32 bits.
__host__ __device__ constexpr int blocks_of(int cols) { return cols / 128 + (cols % 128 != 0); }

constexpr int kDtBf16 = 0, kDtF32 = 1;  // moe_dtype; the third is fp16

template <int DT>
struct Elem;
template <>
struct Elem<0> {
  using type = uint16_t;
};
template <>
struct Elem<1> {
  using type = float;
};
template <>
struct Elem<2> {
  using type = uint16_t;
};

template <int DT>
__device__ __forceinline__ void load16(const typename Elem<DT>::type* p, float (&v)[16]) {
  if constexpr (DT == kDtF32) {
    const float4* q = reinterpret_cast<const float4*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 f = q[i];
      v[4 * i] = f.x;
      v[4 * i + 1] = f.y;
      v[4 * i + 2] = f.z;
      v[4 * i + 3] = f.w;
    }
  } else {
    const uint4* q = reinterpret_cast<const uint4*>(p);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 u = q[i];
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (DT == kDtBf16) {
          v[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
          v[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        } else {
          v[8 * i + 2 * j] = f16_to_f32(static_cast<uint16_t>(w[j]));
          v[8 * i + 2 * j + 1] = f16_to_f32(static_cast<uint16_t>(w[j] >> 16));
        }
      }
    }
  }
}

// The largest |v| as its fp32 bits: they order like the values, and a NaN or
// an infinity shows as bits >= 0x7f800000 (a float maximum would drop NaN).
__device__ __forceinline__ uint32_t amax_bits(const float (&v)[16]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  return m;
}

__device__ __forceinline__ float block_scale(uint32_t bits, int pow2) {
  float s = __uint_as_float(bits) / 448.0f;
  if (pow2) s = __uint_as_float((__float_as_uint(s) + 0x7fffffu) & 0x7f800000u);
  return fmaxf(s, 0x1p-126f);
}

__device__ __forceinline__ uint4 to_codes(const float (&v)[16], float inv) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i] * inv, v[4 * i + 1] * inv, 0, false);
    w[i] = __builtin_amdgcn_cvt_pk_fp8_f32(v[4 * i + 2] * inv, v[4 * i + 3] * inv, r, true);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// z / (1 + e^-z), the quotient from a reciprocal and set right by its residual
// (exact in one FMA): the division's own rounding but for the rarest near
// ties. z = inf gives NaN for inf, which a block takes alike. Below z = -64,
// where the reciprocal of 1 + e^-z would leave the normal range, the division.
__device__ __forceinline__ float silu_quotient(float z) {
  const float d = 1.0f + expf(-z);
  if (z <= -64.0f) return z / d;
  const float r = __builtin_amdgcn_rcpf(d), q = z * r;
  return fmaf(fmaf(-d, q, z), r, q);
}

// Quantise one lane's part of a block whose maximum is `bits` on every lane.
__device__ __forceinline__ uint4 finish(const float (&v)[16], uint32_t bits, int pow2, float* s, int32_t* err) {
  if (bits >= 0x7f800000u) {
    *s = __uint_as_float(0x7fc00000u);
    set_device_error(err, 8);
    return make_uint4(0, 0, 0, 0);
  }
  *s = block_scale(bits, pow2);
  return to_codes(v, 1.0f / *s);
}

// 1 x 128 blocks: 8 lanes per block. SWIGLU: src holds rows of gate | up.
template <int DT, bool SWIGLU>
__global__ __launch_bounds__(256) void k_quantize_rows(const typename Elem<DT>::type* __restrict__ src, int64_t rows,
                                                       int cols, int pow2, uint8_t* __restrict__ codes,
                                                       float* __restrict__ scales, int32_t* err) {
  const int nb = blocks_of(cols);
  const uint32_t unit = blockIdx.x * 32 + threadIdx.x / 8;  // block of 128; a grid holds fewer than 2^24 workgroups
  const int64_t row = unit / static_cast<uint32_t>(nb);
  const int b = static_cast<int>(unit % static_cast<uint32_t>(nb));
  const int c = b * 128 + (threadIdx.x & 7) * 16;
  const bool valid = row < rows && c < cols;  // the lanes past the end stay in the shuffles
  float v[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = 0.0f;
  if (valid) {
    if constexpr (SWIGLU) {
      float u[16];
      const typename Elem<DT>::type* p = src + row * (2 * static_cast<int64_t>(cols)) + c;
      load16<DT>(p, v);
      load16<DT>(p + cols, u);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = silu_quotient(v[i]) * u[i];
    } else {
      load16<DT>(src + row * cols + c, v);
    }
  }
  uint32_t bits = amax_bits(v);
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) bits = max(bits, static_cast<uint32_t>(__shfl_xor(static_cast<int>(bits), o)));
  if (!valid) return;
  float s;
  const uint4 q = finish(v, bits, pow2, &s, err);
  *reinterpret_cast<uint4*>(codes + row * cols + c) = q;
  if ((threadIdx.x & 7) == 0) scales[unit] = s;
}

// 128 x 128 blocks: one workgroup per block, each lane 16 columns of 4 rows.
template <int DT>
__global__ __launch_bounds__(256) void k_quantize_tiles(const typename Elem<DT>::type* __restrict__ src, int64_t rows,
                                                        int cols, int64_t row_blocks, int pow2,
                                                        uint8_t* __restrict__ codes, float* __restrict__ scales,
                                                        int32_t* err) {
  __shared__ uint32_t s_max[4];
  const int nb = blocks_of(cols);
  const int64_t tile = blockIdx.x;
  const int64_t mr = tile / nb;  // matrix * row_blocks + row block
  const int64_t m = mr / row_blocks;
  const int64_t r0 = (mr - m * row_blocks) * 128 + threadIdx.x / 8;
  const int c = static_cast<int>(tile - mr * nb) * 128 + (threadIdx.x & 7) * 16;
  float v[4][16];
  uint32_t bits = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int j = 0; j < 16; ++j) v[i][j] = 0.0f;
    if (c < cols && r0 + 32 * i < rows) load16<DT>(src + (m * rows + r0 + 32 * i) * cols + c, v[i]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) bits = max(bits, amax_bits(v[i]));
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) bits = max(bits, static_cast<uint32_t>(__shfl_xor(static_cast<int>(bits), o)));
  if (lane_id() == 0) s_max[threadIdx.x / 64] = bits;
  __syncthreads();
  bits = max(max(s_max[0], s_max[1]), max(s_max[2], s_max[3]));
  float s;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 q = finish(v[i], bits, pow2, &s, err);
    if (c < cols && r0 + 32 * i < rows)
      *reinterpret_cast<uint4*>(codes + (m * rows + r0 + 32 * i) * cols + c) = q;
  }
  if (threadIdx.x == 0) scales[tile] = s;
}

template <int DT, bool SWIGLU>
hipError_t launch_rows(const void* x, int64_t rows, int cols, int pow2, uint8_t* codes, float* scales, int32_t* err,
                       hipStream_t s) {
  const int64_t groups = (rows * blocks_of(cols) + 31) / 32;
  if (groups > max_workgroups(256)) return hipErrorInvalidValue;
  QSMOE_LAUNCH((k_quantize_rows<DT, SWIGLU>), dim3(static_cast<unsigned>(groups)), dim3(256), 0, s,
               static_cast<const typename Elem<DT>::type*>(x), rows, cols, pow2, codes, scales, err);
  return hipGetLastError();
}

template <int DT>
hipError_t launch_tiles(const void* x, int64_t matrices, int64_t rows, int cols, int pow2, uint8_t* codes,
                        float* scales, int32_t* err, hipStream_t s) {
  const int64_t rb = (rows + 127) / 128, nb = blocks_of(cols);
  constexpr int64_t most = max_workgroups(256);
  if (matrices > most / rb || matrices * rb > most / nb) return hipErrorInvalidValue;
  QSMOE_LAUNCH((k_quantize_tiles<DT>), dim3(static_cast<unsigned>(matrices * rb * nb)), dim3(256), 0, s,
               static_cast<const typename Elem<DT>::type*>(x), rows, cols, rb, pow2, codes, scales, err);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quantize_block(const void* x, int dtype, int64_t matrices, int64_t rows, int cols, int block_rows,
                                 int pow2, uint8_t* codes, float* scales, int32_t* err, hipStream_t s) {
  if (block_rows == 1) {
    switch (dtype) {
      case 0: return launch_rows<0, false>(x, matrices * rows, cols, pow2, codes, scales, err, s);
      case 1: return launch_rows<1, false>(x, matrices * rows, cols, pow2, codes, scales, err, s);
      default: return launch_rows<2, false>(x, matrices * rows, cols, pow2, codes, scales, err, s);
    }
  }
  switch (dtype) {
    case 0: return launch_tiles<0>(x, matrices, rows, cols, pow2, codes, scales, err, s);
    case 1: return launch_tiles<1>(x, matrices, rows, cols, pow2, codes, scales, err, s);
    default: return launch_tiles<2>(x, matrices, rows, cols, pow2, codes, scales, err, s);
  }
}

hipError_t launch_swiglu_quantize_block(const void* gu, int dtype, int64_t rows, int inner, int pow2, uint8_t* codes,
                                        float* scales, int32_t* err, hipStream_t s) {
  switch (dtype) {
    case 0: return launch_rows<0, true>(gu, rows, inner, pow2, codes, scales, err, s);
    case 1: return launch_rows<1, true>(gu, rows, inner, pow2, codes, scales, err, s);
    default: return launch_rows<2, true>(gu, rows, inner, pow2, codes, scales, err, s);
  }
}

}  // namespace qsmoe

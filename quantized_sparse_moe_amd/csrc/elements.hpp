// Rows of bf16, fp32 or fp16 elements, eight at a time, at any alignment of
// their first element, for the kernels that move and weight whole rows.
#pragma once

#include <type_traits>

#include "common.hpp"

namespace qsmoe {

constexpr int kBf16 = 0, kF32 = 1, kF16 = 2;  // moe_dtype

template <int DT>
constexpr int kElemBytes = DT == kF32 ? 4 : 2;

// Eight elements as 32-bit words. Rows of an odd length start at any element,
// so the vectors promise no more than an element's alignment: one 16-byte
// access each all the same, as the hardware takes unaligned global addresses.
typedef __attribute__((ext_vector_type(4))) uint32_t words4_t;
typedef __attribute__((ext_vector_type(4), aligned(2))) uint32_t words4_any2_t;
typedef __attribute__((ext_vector_type(4), aligned(4))) uint32_t words4_any4_t;

template <int DT>
struct Raw8 {
  words4_t w[DT == kF32 ? 2 : 1];
};

template <int DT>
__device__ __forceinline__ Raw8<DT> load_raw8(const char* p) {
  Raw8<DT> r;
  if constexpr (DT == kF32) {
    r.w[0] = *reinterpret_cast<const words4_any4_t*>(p);
    r.w[1] = *reinterpret_cast<const words4_any4_t*>(p + 16);
  } else {
    r.w[0] = *reinterpret_cast<const words4_any2_t*>(p);
  }
  return r;
}

template <int DT>
__device__ __forceinline__ void store_raw8(char* p, const Raw8<DT>& r) {
  if constexpr (DT == kF32) {
    *reinterpret_cast<words4_any4_t*>(p) = r.w[0];
    *reinterpret_cast<words4_any4_t*>(p + 16) = r.w[1];
  } else {
    *reinterpret_cast<words4_any2_t*>(p) = r.w[0];
  }
}

// The first n < 8 elements, zeros behind them.
template <int DT>
__device__ __forceinline__ Raw8<DT> load_raw_part(const char* p, int n) {
  Raw8<DT> r{};
#pragma unroll
  for (int i = 0; i < 7; ++i) {
    if (i < n) {
      if constexpr (DT == kF32)
        r.w[i / 4][i % 4] = reinterpret_cast<const uint32_t*>(p)[i];
      else
        r.w[0][i / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p)[i]) << (16 * (i % 2));
    }
  }
  return r;
}

template <int DT>
__device__ __forceinline__ void store_raw_part(char* p, const Raw8<DT>& r, int n) {
#pragma unroll
  for (int i = 0; i < 7; ++i) {
    if (i < n) {
      if constexpr (DT == kF32)
        reinterpret_cast<uint32_t*>(p)[i] = r.w[i / 4][i % 4];
      else
        reinterpret_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(r.w[0][i / 2] >> (16 * (i % 2)));
    }
  }
}

// n: elements that exist from p on.
template <int DT>
__device__ __forceinline__ Raw8<DT> load_raw(const char* p, int n) {
  return n >= 8 ? load_raw8<DT>(p) : load_raw_part<DT>(p, n);
}
template <int DT>
__device__ __forceinline__ void store_raw(char* p, const Raw8<DT>& r, int n) {
  if (n >= 8)
    store_raw8<DT>(p, r);
  else
    store_raw_part<DT>(p, r, n);
}

template <int DT>
__device__ __forceinline__ void to_f32(const Raw8<DT>& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if constexpr (DT == kF32) {
      v[i] = __uint_as_float(r.w[i / 4][i % 4]);
    } else {
      const uint32_t w = r.w[0][i / 2];
      if constexpr (DT == kBf16)
        v[i] = __uint_as_float(i % 2 ? w & 0xffff0000u : w << 16);
      else
        v[i] = f16_to_f32(static_cast<uint16_t>(i % 2 ? w >> 16 : w));
    }
  }
}

// Rounded once, to the nearest even.
template <int DT>
__device__ __forceinline__ Raw8<DT> from_f32(const float (&v)[8]) {
  Raw8<DT> r;
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    if constexpr (DT == kF32) {
      r.w[i / 4][i % 4] = __float_as_uint(v[i]);
      r.w[i / 4][i % 4 + 1] = __float_as_uint(v[i + 1]);
    } else if constexpr (DT == kBf16) {
      bf16x2_t p;
      p[0] = static_cast<__bf16>(v[i]);
      p[1] = static_cast<__bf16>(v[i + 1]);
      r.w[0][i / 2] = __builtin_bit_cast(uint32_t, p);
    } else {
      const uint32_t lo = __builtin_bit_cast(uint16_t, static_cast<_Float16>(v[i]));
      const uint32_t hi = __builtin_bit_cast(uint16_t, static_cast<_Float16>(v[i + 1]));
      r.w[0][i / 2] = lo | (hi << 16);
    }
  }
  return r;
}

// How a workgroup of 256 lanes is laid over rows of `vectors` eights: 2^shift
// lanes to a row, `chunks` workgroups to one row where 256 lanes do not reach.
struct RowSplit {
  int32_t shift, chunks;
  int64_t blocks;
};
inline RowSplit split_rows(int64_t rows, int64_t elements) {
  const int64_t vectors = (elements + 7) / 8;
  RowSplit s{0, 1, 0};
  while (s.shift < 8 && (int64_t{1} << s.shift) < vectors) ++s.shift;
  s.chunks = static_cast<int32_t>((vectors + 255) / 256);
  if (s.chunks < 1) s.chunks = 1;
  const int64_t per_block = 256 >> s.shift;
  s.blocks = (rows + per_block - 1) / per_block * s.chunks;
  return s;
}
// This lane's row and first element in block b.
__device__ __forceinline__ void place_of(const RowSplit& s, int64_t b, int64_t* row, int* at) {
  const int64_t group = s.chunks == 1 ? b : b / s.chunks;
  const int chunk = static_cast<int>(b - group * s.chunks);
  *row = group * (256 >> s.shift) + (threadIdx.x >> s.shift);
  *at = 8 * ((chunk << s.shift) + (threadIdx.x & ((1 << s.shift) - 1)));
}

// A grid for `blocks` workgroups of 256 that step on by the grid.
inline unsigned grid_of(int64_t blocks) {
  constexpr int64_t most = (int64_t{1} << 24) - 8;  // HIP counts a grid's threads with 32 bits
  return static_cast<unsigned>(blocks < most ? blocks : most);
}

// Calls f with an element type as a constant.
template <typename F>
inline hipError_t with_type(int dtype, F f) {
  switch (dtype) {
    case kBf16: return f(std::integral_constant<int, kBf16>{});
    case kF32: return f(std::integral_constant<int, kF32>{});
    default: return f(std::integral_constant<int, kF16>{});
  }
}

}  // namespace qsmoe

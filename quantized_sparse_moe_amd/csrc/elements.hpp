// Rows of bf16, fp32 or fp16 elements, eight at a time, at any alignment of
// their first element, for the kernels that move and weight whole rows.
#pragma once

#include <type_traits>

#include "common.hpp"

namespace qsmoe {

constexpr int kBf16 = 0, kF32 = 1, kF16 = 2;  // moe_dtype

template <int DT>
constexpr int kElemBytes = DT == kF32 ? 4 : 2;

// V elements, 4 or 8, as 32-bit words: 8 of the 16-bit types or 4 of fp32 are
// one access of 16 bytes. Rows of an odd length start at any element, so the
// vectors promise no more than an element's alignment; the hardware takes
// unaligned global addresses in one access all the same.
template <int DT, int V>
struct Raw {
  static constexpr int kWords = V * kElemBytes<DT> / 4, kVector = kWords < 4 ? kWords : 4;
  typedef __attribute__((ext_vector_type(kVector), aligned(kElemBytes<DT>))) uint32_t any_t;
  uint32_t w[kWords];
};

// How many elements a lane takes at a time where rows of types A and B meet: a
// lane's part of an fp32 row is one access, so that a wave's accesses cover
// whole lines.
template <int A, int B>
constexpr int kLaneElems = A == kF32 || B == kF32 ? 4 : 8;

// The first n < V elements, zeros behind them.
template <int DT, int V>
__device__ __forceinline__ Raw<DT, V> load_part(const char* p, int n) {
  Raw<DT, V> r{};
#pragma unroll
  for (int i = 0; i < V - 1; ++i) {
    if (i < n) {
      if constexpr (DT == kF32)
        r.w[i] = reinterpret_cast<const uint32_t*>(p)[i];
      else
        r.w[i / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p)[i]) << (16 * (i % 2));
    }
  }
  return r;
}

template <int DT, int V>
__device__ __forceinline__ void store_part(char* p, const Raw<DT, V>& r, int n) {
#pragma unroll
  for (int i = 0; i < V - 1; ++i) {
    if (i < n) {
      if constexpr (DT == kF32)
        reinterpret_cast<uint32_t*>(p)[i] = r.w[i];
      else
        reinterpret_cast<uint16_t*>(p)[i] = static_cast<uint16_t>(r.w[i / 2] >> (16 * (i % 2)));
    }
  }
}

// V elements, of which n exist from p on.
template <int DT, int V>
__device__ __forceinline__ Raw<DT, V> load_raw(const char* p, int n) {
  if (n < V) return load_part<DT, V>(p, n);
  using R = Raw<DT, V>;
  R r;
#pragma unroll
  for (int i = 0; i < R::kWords; i += R::kVector) {
    const auto v = *reinterpret_cast<const typename R::any_t*>(p + 4 * i);
#pragma unroll
    for (int j = 0; j < R::kVector; ++j) r.w[i + j] = v[j];
  }
  return r;
}

// ONCE: past the caches, for results larger than they are.
template <int DT, int V, bool ONCE = false>
__device__ __forceinline__ void store_raw(char* p, const Raw<DT, V>& r, int n) {
  if (n < V) return store_part<DT, V>(p, r, n);
  using R = Raw<DT, V>;
#pragma unroll
  for (int i = 0; i < R::kWords; i += R::kVector) {
    typename R::any_t v;
#pragma unroll
    for (int j = 0; j < R::kVector; ++j) v[j] = r.w[i + j];
    if constexpr (ONCE)
      __builtin_nontemporal_store(v, reinterpret_cast<typename R::any_t*>(p + 4 * i));
    else
      *reinterpret_cast<typename R::any_t*>(p + 4 * i) = v;
  }
}

template <int DT, int V>
__device__ __forceinline__ void to_f32(const Raw<DT, V>& r, float (&v)[V]) {
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if constexpr (DT == kF32) {
      v[i] = __uint_as_float(r.w[i]);
    } else {
      const uint32_t w = r.w[i / 2];
      if constexpr (DT == kBf16)
        v[i] = __uint_as_float(i % 2 ? w & 0xffff0000u : w << 16);
      else
        v[i] = f16_to_f32(static_cast<uint16_t>(i % 2 ? w >> 16 : w));
    }
  }
}

// Rounded once, to the nearest even.
template <int DT, int V>
__device__ __forceinline__ Raw<DT, V> from_f32(const float (&v)[V]) {
  Raw<DT, V> r;
#pragma unroll
  for (int i = 0; i < V; i += 2) {
    if constexpr (DT == kF32) {
      r.w[i] = __float_as_uint(v[i]);
      r.w[i + 1] = __float_as_uint(v[i + 1]);
    } else if constexpr (DT == kBf16) {
      bf16x2_t p;
      p[0] = static_cast<__bf16>(v[i]);
      p[1] = static_cast<__bf16>(v[i + 1]);
      r.w[i / 2] = __builtin_bit_cast(uint32_t, p);
    } else {
      const uint32_t lo = __builtin_bit_cast(uint16_t, static_cast<_Float16>(v[i]));
      const uint32_t hi = __builtin_bit_cast(uint16_t, static_cast<_Float16>(v[i + 1]));
      r.w[i / 2] = lo | (hi << 16);
    }
  }
  return r;
}

// How a workgroup of 256 lanes is laid over rows, V elements a lane: 2^shift
// lanes to a row, `chunks` workgroups to one row where 256 lanes do not reach.
struct RowSplit {
  int32_t shift, chunks;
  int64_t blocks;
};
inline RowSplit split_rows(int64_t rows, int64_t elements, int V) {
  const int64_t vectors = (elements + V - 1) / V;
  RowSplit s{0, 1, 0};
  while (s.shift < 8 && (int64_t{1} << s.shift) < vectors) ++s.shift;
  s.chunks = static_cast<int32_t>((vectors + 255) / 256);
  if (s.chunks < 1) s.chunks = 1;
  const int64_t per_block = 256 >> s.shift;
  s.blocks = (rows + per_block - 1) / per_block * s.chunks;
  return s;
}
// This lane's row and first element in block b.
template <int V>
__device__ __forceinline__ void place_of(const RowSplit& s, int64_t b, int64_t* row, int* at) {
  const int64_t group = s.chunks == 1 ? b : b / s.chunks;
  const int chunk = static_cast<int>(b - group * s.chunks);
  *row = group * (256 >> s.shift) + (threadIdx.x >> s.shift);
  *at = V * ((chunk << s.shift) + (threadIdx.x & ((1 << s.shift) - 1)));
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

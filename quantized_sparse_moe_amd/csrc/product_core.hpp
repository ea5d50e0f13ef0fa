// Device-side parts of the matrix-core products grouped by expert.
#pragma once

#include "common.hpp"
#include "kernels.hpp"

namespace qsmoe {

typedef __attribute__((ext_vector_type(8))) __bf16 bf16x8_t;
typedef __attribute__((ext_vector_type(8))) _Float16 f16x8_t;
typedef __attribute__((ext_vector_type(4))) float f32x4_t;
typedef __attribute__((ext_vector_type(4))) uint32_t u32x4_t;
typedef __attribute__((ext_vector_type(8))) int i32x8_t;

typedef __attribute__((address_space(1))) void global_void_t;
typedef __attribute__((address_space(3))) void lds_void_t;
typedef __attribute__((address_space(3))) u32x4_t lds_u32x4_t;

enum : int { kBucket = 0, kToken = 1, kSlot = 2 };  // moe_rows

// The row of a matrix in `order` that belongs to a bucket position, from the
// position (bucket order) or perm's entry for it; -1 where perm holds no
// assignment (which sets the error bit).
__device__ __forceinline__ int row_in(int a, int order, int k, int n, int32_t* err) {
  if (order == kBucket) return a;
  if (a < 0 || a >= n) {
    set_device_error(err, 16);
    return -1;
  }
  return order == kToken ? a / k : a;
}
__device__ __forceinline__ int row_of(const int32_t* perm, int order, int k, int n, int p, int32_t* err) {
  return row_in(order == kBucket ? p : perm[p], order, k, n, err);
}

// Direct global -> LDS load of 16 bytes per lane: lane l's bytes land at
// lds + 16 l, lds being the same for the whole wave. Counted by vmcnt.
__device__ __forceinline__ void load_lds16(const void* src, char* lds) {
  __builtin_amdgcn_global_load_lds((global_void_t*)(src), (lds_void_t*)(lds), 16, 0, 0);
}
__device__ __forceinline__ void load_lds4(const void* src, char* lds) {
  __builtin_amdgcn_global_load_lds((global_void_t*)(src), (lds_void_t*)(lds), 4, 0, 0);
}

// Workgroup barrier that leaves the wave's N newest vector loads in flight:
// loads complete in order, so everything older has landed in LDS. Fences for
// the compiler only: a release fence would wait for every load.
template <int N>
__device__ __forceinline__ void barrier_keep() {
  static_assert(N >= 0 && N < 16, "low vmcnt field");
  __builtin_amdgcn_s_waitcnt(0x0070 | N);  // vmcnt(N) lgkmcnt(0)
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
  __builtin_amdgcn_s_barrier();
  __atomic_signal_fence(__ATOMIC_SEQ_CST);
}

__device__ __forceinline__ u32x4_t lds16(const char* p) { return *(const lds_u32x4_t*)(p); }

// Four fragments of an operand stored across the contraction, by transposing
// LDS reads: 16 lanes address a 4 x 16 square of 16-bit values (lane i: row
// i / 4, columns 4 (i % 4) .. + 3) and lane i gets column i. Each fragment
// takes the squares at offsets LO and HI behind its address. In assembly with
// the wait in the same block: for the builtin the compiler would also wait for
// every direct-to-LDS load in flight.
template <int LO, int HI>
__device__ __forceinline__ void lds_tr_x4(const int (&at)[4], u32x4_t (&f)[4]) {
  static_assert(LO >= 0 && HI < 65536, "16-bit LDS offset");
  typedef __attribute__((ext_vector_type(2))) uint32_t u32x2_t;
  u32x2_t o0, o1, o2, o3, o4, o5, o6, o7;
  asm volatile(
      "ds_read_b64_tr_b16 %0, %8 offset:%12\n"
      "ds_read_b64_tr_b16 %1, %8 offset:%13\n"
      "ds_read_b64_tr_b16 %2, %9 offset:%12\n"
      "ds_read_b64_tr_b16 %3, %9 offset:%13\n"
      "ds_read_b64_tr_b16 %4, %10 offset:%12\n"
      "ds_read_b64_tr_b16 %5, %10 offset:%13\n"
      "ds_read_b64_tr_b16 %6, %11 offset:%12\n"
      "ds_read_b64_tr_b16 %7, %11 offset:%13\n"
      "s_waitcnt lgkmcnt(0)"
      : "=&v"(o0), "=&v"(o1), "=&v"(o2), "=&v"(o3), "=&v"(o4), "=&v"(o5), "=&v"(o6), "=&v"(o7)
      : "v"(at[0]), "v"(at[1]), "v"(at[2]), "v"(at[3]), "i"(LO), "i"(HI)
      : "memory");
  f[0] = __builtin_shufflevector(o0, o1, 0, 1, 2, 3);
  f[1] = __builtin_shufflevector(o2, o3, 0, 1, 2, 3);
  f[2] = __builtin_shufflevector(o4, o5, 0, 1, 2, 3);
  f[3] = __builtin_shufflevector(o6, o7, 0, 1, 2, 3);
}
__device__ __forceinline__ int lds_address(const char* p) {
  return static_cast<int>(reinterpret_cast<uintptr_t>((const __attribute__((address_space(3))) char*)(p)));
}

template <int TYPE>
__device__ __forceinline__ f32x4_t mma16(u32x4_t a, u32x4_t b, f32x4_t c) {
  if constexpr (TYPE == 0)
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c,
                                                   0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0,
                                                  0, 0);
}

// 16 x 16 x 128 over E4M3 from zero; the unscaled form (scales 0). The
// instruction sums 8 neighbouring products at a time on the exponent of the
// largest and drops what lies more than 13 bits below it (measured: a second
// product is exact down to 2^-13 of the first, changed from 2^-14 on, and lost
// too where the largest products cancel; groups of 8 are then summed in fp32).
// The error is at most 7 * 2^-13 of the largest product of a group. Measured
// over blocks of 128, as a share of the result in the norm: normal inputs
// 1.3e-5, inputs of one sign 3.0e-6 (2.4e-6 of it towards zero), channels
// scaled by e^(2 z) 5.3e-5, the largest error of one result 1.9e-4 of its sum
// of |products|. Rounding to bf16 is 1.66e-3 in the norm, 30 times the worst of
// these, so bf16 outputs are formed this way unless the caller asks for fp32
// sums (their error against 64 bits is 1.6595e-3, of which rounding alone makes
// 1.6594e-3). Rounding to fp16, 2.1e-4, is not far enough above it: fp16 and
// fp32 outputs go through bf16, where every product is exact and sums are fp32
// (1e-8 to 4e-8 in the same three norms). The K = 32 FP8 instruction drops the
// same bits.
__device__ __forceinline__ f32x4_t mma_fp8(i32x8_t a, i32x8_t b) {
  const f32x4_t z = {0.0f, 0.0f, 0.0f, 0.0f};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, z, 0, 0, 0, 0, 0, 0);
}

// 8 E4M3 codes as bf16 (exact).
__device__ __forceinline__ u32x4_t e4m3_to_bf16x8(uint32_t a, uint32_t b) {
  u32x4_t r;
  r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, false));
  r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(a, 1.0f, true));
  r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, false));
  r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(b, 1.0f, true));
  return r;
}

// Store 4 consecutive outputs (8- or 16-byte aligned).
__device__ __forceinline__ uint32_t pack2(int out_type, float a, float b) {
  if (out_type == 0) return f32_to_bf16_rne(a) | (f32_to_bf16_rne(b) << 16);
  const uint32_t lo = __builtin_bit_cast(uint16_t, static_cast<_Float16>(a));
  const uint32_t hi = __builtin_bit_cast(uint16_t, static_cast<_Float16>(b));
  return lo | (hi << 16);
}
__device__ __forceinline__ void store4(char* p, int out_type, f32x4_t v) {
  if (out_type == 1) {
    *reinterpret_cast<f32x4_t*>(p) = v;
  } else {
    uint2 u;
    u.x = pack2(out_type, v[0], v[1]);
    u.y = pack2(out_type, v[2], v[3]);
    *reinterpret_cast<uint2*>(p) = u;
  }
}

__device__ __forceinline__ void store8(char* p, int out_type, f32x4_t v, f32x4_t w) {
  if (out_type == 1) {
    reinterpret_cast<f32x4_t*>(p)[0] = v;
    reinterpret_cast<f32x4_t*>(p)[1] = w;
  } else {
    uint4 u;
    u.x = pack2(out_type, v[0], v[1]);
    u.y = pack2(out_type, v[2], v[3]);
    u.z = pack2(out_type, w[0], w[1]);
    u.w = pack2(out_type, w[2], w[3]);
    *reinterpret_cast<uint4*>(p) = u;
  }
}

// fp32 results of two neighbouring 16 x 16 fragments, whole 128-byte lines at
// a time: lane (g, j) holds columns 4 g .. + 3 of both in row j; lanes j and
// j ^ 8 trade, so that the first store writes 32 columns of rows 0 .. 7 and
// the second those of rows 8 .. 15. row_ptr(r): address of the first
// fragment's first column in row r, or null; left: columns that exist.
template <typename F>
__device__ __forceinline__ void store_pair_f32(f32x4_t f0, f32x4_t f1, int left, F row_ptr) {
  const int lane = lane_id(), g = lane >> 4, j = lane & 15;
  const bool low = j < 8;
  f32x4_t first, second;
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    const float traded = __int_as_float(
        __builtin_amdgcn_update_dpp(0, __float_as_int(low ? f1[v] : f0[v]), 0x128, 0xf, 0xf, true));  // row_ror:8
    first[v] = low ? f0[v] : traded;
    second[v] = low ? traded : f1[v];
  }
  const int c = (low ? 0 : 16) + 4 * g;
  if (c >= left) return;
  float* p = row_ptr(j & 7);
  if (p) *reinterpret_cast<f32x4_t*>(p + c) = first;
  p = row_ptr(8 + (j & 7));
  if (p) *reinterpret_cast<f32x4_t*>(p + c) = second;
}

// Inclusive sum over the wave's lanes: rows of 16 by DPP shifts, then the row
// totals handed on.
__device__ __forceinline__ int wave_scan(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, true);  // row_shr:1
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, true);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, true);  // row_bcast:15 into rows 1 and 3
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, true);  // row_bcast:31 into rows 2 and 3
  return v;
}

// Tile `pair` of the list of every expert's (row tile, column tile) pairs.
// Each wave finds it by itself, without LDS or a barrier: 4 experts a lane,
// their tile counts scanned across the lanes, 256 experts at a time. Within an
// expert row tiles run fastest, in bands of 8, so that the workgroups of one
// XCD share both a band's rows and few column tiles (bf16 8192^3: 818 us, in
// bands of 4 822, of 16 870).
struct TileAt {
  int e, first, rows, ctile;
};
template <int BM>
__device__ __forceinline__ bool find_tile(const int32_t* offsets, int E, int n, int ctiles, int64_t pair, TileAt* t) {
  int64_t before = 0;
  int e = 0, lo = 0, count = n;
  if (offsets) {
    const int lane = lane_id();
    bool found = false;
    for (int e0 = 0; e0 < E; e0 += 256) {
      const int i = e0 + 4 * lane;
      int o[5], mt[4];
#pragma unroll
      for (int v = 0; v < 5; ++v) o[v] = min(max(offsets[min(i + v, E)], 0), n);
      int sum = 0;
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        mt[v] = (max(o[v + 1] - o[v], 0) + BM - 1) / BM;  // 0 past the last expert
        sum += mt[v];
      }
      const int incl = wave_scan(sum);
      const uint64_t m = __ballot(before + static_cast<int64_t>(incl) * ctiles > pair);
      if (m != 0) {
        const int src = __ffsll(static_cast<unsigned long long>(m)) - 1;
        before += static_cast<int64_t>(__builtin_amdgcn_readlane(incl - sum, src)) * ctiles;
        e = e0 + 4 * src;
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          const int64_t here = static_cast<int64_t>(__builtin_amdgcn_readlane(mt[v], src)) * ctiles;
          if (!found) {
            if (before + here > pair) {
              found = true;
              e += v;
              lo = __builtin_amdgcn_readlane(o[v], src);
              count = __builtin_amdgcn_readlane(o[v + 1], src) - lo;
            } else {
              before += here;
            }
          }
        }
        break;
      }
      before += static_cast<int64_t>(__builtin_amdgcn_readlane(incl, 63)) * ctiles;
    }
    if (!found) return false;
  } else if (pair >= static_cast<int64_t>((n + BM - 1) / BM) * ctiles) {
    return false;
  }
  const int mt = (count + BM - 1) / BM;
  const int64_t at = pair - before;
  const int64_t band = at / (8 * static_cast<int64_t>(ctiles));
  // never so with buckets that lie side by side; overlapping ones of many
  // millions of rows could wrap the count of tiles
  if (at < 0 || 8 * band >= mt) return false;
  const int high = min(8, mt - 8 * static_cast<int>(band));
  const int rest = static_cast<int>(at - band * 8 * ctiles);
  const int mtile = 8 * static_cast<int>(band) + rest % high;
  t->e = e;
  t->ctile = rest / high;
  if (t->ctile >= ctiles) return false;
  t->first = lo + mtile * BM;
  t->rows = min(count - mtile * BM, BM);
  return true;
}

// Workgroup b runs on XCD b % 8. Pairs go to the XCDs in runs of `run`, so
// that neighbours in the list share an L2 and all XCDs move through the list
// together.
__device__ __forceinline__ int64_t pair_of_block(int run) {
  const unsigned b = blockIdx.x, x = b & 7u, l = b >> 3;
  return static_cast<int64_t>(l / run * 8 + x) * run + l % run;
}

}  // namespace qsmoe

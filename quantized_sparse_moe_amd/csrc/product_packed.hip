// Products of few rows with 4-bit weights, dense or grouped by expert:
//   out[p][n] = sum_k x[p][k] W[n][k],
// W affine (w = s q + b, fp16 s and b per group of 32, 64 or 128) or MXFP4 (w =
// 2^(s - 127) e2m1(q) per 32). Within a group g of a row n
//   sum_k x w = s (sum_k x q) + b (sum_k x),
// so the codes go to the matrix cores as they are, exact in bf16 and fp16, and
// scales and biases touch each group's sum only.
//
// The weights are the right operand of v_mfma_f32_16x16x32: lane (n, q), n =
// lane % 16, q = lane / 16, loads 16 bytes, the 32 codes from 32 q on of row
// n's 128-code chunk, and word i of them is the lane's part of product i. So
// product i takes 8 codes of each quarter of the chunk, and of up to 4 groups.
// The groups stay apart through the left operand: its 16 rows are (row of x,
// group), 4, 8 or 16 rows of x for groups of 32, 64 and 128, and row (t, g)
// holds x_t where the quarter lies in group g and zeros elsewhere. The result's
// layout then gives lane (n, q) the sums of row n for one to four rows of x
// with its groups in order, as the lane holds row n's scales; the sums of x
// come from the same products with a right operand of ones. For one row of x
// three quarters of the products are zeros, but the matrix cores have the time.
#include <algorithm>

#include "elements.hpp"
#include "kernels.hpp"
#include "product_core.hpp"

namespace qsmoe {

namespace {

constexpr int kWaves = 8;
constexpr int kChunk = 128;

// Four words of 8 codes each as matrix operands: affine codes 8 by 8 in the
// order 0 2 4 6 1 3 5 7. A nibble n as an E4M3 byte is n * 2^-9, the
// conversion's scale makes it n.
template <int TYPE, int FMT>
__device__ __forceinline__ u32x4_t codes_to_16(uint32_t w) {
  u32x4_t r;
  if constexpr (FMT == 0) {
    const uint32_t even = w & 0x0f0f0f0fu, odd = (w >> 4) & 0x0f0f0f0fu;
    if constexpr (TYPE == kBf16) {
      r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(even, 512.0f, false));
      r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(even, 512.0f, true));
      r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(odd, 512.0f, false));
      r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(odd, 512.0f, true));
    } else {
      r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(even, 512.0f, false));
      r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(even, 512.0f, true));
      r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(odd, 512.0f, false));
      r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(odd, 512.0f, true));
    }
  } else if constexpr (TYPE == kBf16) {
    r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 0));
    r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 1));
    r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 2));
    r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 3));
  } else {
    r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0));
    r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1));
    r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2));
    r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3));
  }
  return r;
}

// 8 values of x in the order of the codes.
template <int FMT>
__device__ __forceinline__ u32x4_t in_code_order(u32x4_t x) {
  if constexpr (FMT != 0) return x;
  u32x4_t r;
  r[0] = __builtin_amdgcn_perm(x[1], x[0], 0x05040100u);
  r[1] = __builtin_amdgcn_perm(x[3], x[2], 0x05040100u);
  r[2] = __builtin_amdgcn_perm(x[1], x[0], 0x07060302u);
  r[3] = __builtin_amdgcn_perm(x[3], x[2], 0x07060302u);
  return r;
}

template <int CTRL>
__device__ __forceinline__ u32x4_t quad_moved(u32x4_t v, uint32_t mask) {
  u32x4_t r;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    r[j] = static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v[j]), CTRL, 0xf, 0xf, true)) & mask;
  return r;
}

// The scales of a chunk's NG groups of one row, packed as they lie.
template <int FMT, int NG>
struct Packed {
  using type = std::conditional_t<FMT == 1 || NG == 2, uint32_t, std::conditional_t<NG == 4, uint64_t, uint16_t>>;
};
template <int FMT, int NG>
using packed_t = typename Packed<FMT, NG>::type;

// Groups first .. first + NG - 1 of a row of G; zeros past its end. Rows lie at
// any element, so the load promises no more.
template <int FMT, int NG>
__device__ __forceinline__ packed_t<FMT, NG> load_groups(const char* row, int first, int G) {
  constexpr int kSize = FMT == 0 ? 2 : 1;
  using P = packed_t<FMT, NG>;
  if (G >= NG) {
    const int from = min(first, G - NG);
    typedef P __attribute__((aligned(FMT == 0 ? 2 : 1))) any_t;
    const P v = *reinterpret_cast<const any_t*>(row + from * kSize);
    return static_cast<P>(v >> (8 * kSize * (first - from)));
  }
  P v = 0;
  for (int i = 0; i < G; ++i) {
    const P one = FMT == 0 ? reinterpret_cast<const uint16_t*>(row)[i] : reinterpret_cast<const uint8_t*>(row)[i];
    v |= static_cast<P>(one << (8 * kSize * i));
  }
  return v;
}

template <int FMT, int NG>
__device__ __forceinline__ float group_scale(packed_t<FMT, NG> v, int g) {
  if constexpr (FMT == 0)
    return f16_to_f32(static_cast<uint16_t>(v >> (16 * g)));
  else
    return e8m0_to_f32(static_cast<uint32_t>(v >> (8 * g)) & 0xffu);
}

// The b-th expert with rows and its positions, offsets clamped to [0, n].
// Uniform over the wave: 4 experts a lane, their count scanned.
__device__ __forceinline__ bool find_bucket(const int32_t* offsets, int E, int n, int b, int* e, int* lo, int* hi) {
  const int lane = lane_id();
  int before = 0;
  for (int e0 = 0; e0 < E; e0 += 256) {
    const int i = e0 + 4 * lane;
    int o[5], sum = 0;
#pragma unroll
    for (int v = 0; v < 5; ++v) o[v] = min(max(offsets[min(i + v, E)], 0), n);
#pragma unroll
    for (int v = 0; v < 4; ++v) sum += o[v + 1] > o[v];
    const int incl = wave_scan(sum);
    const uint64_t m = __ballot(before + incl > b);
    if (m != 0) {
      const int src = __ffsll(static_cast<unsigned long long>(m)) - 1;
      int at = before + __builtin_amdgcn_readlane(incl - sum, src);
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int from = __builtin_amdgcn_readlane(o[v], src), to = __builtin_amdgcn_readlane(o[v + 1], src);
        if (to > from && at++ == b) {
          *e = e0 + 4 * src + v;
          *lo = from;
          *hi = to;
          return true;
        }
      }
    }
    before += __builtin_amdgcn_readlane(incl, 63);
  }
  return false;
}

// A tile is 16 rows of W; kw of the workgroup's 8 waves share its contraction.
// AB left operands, AB * 16 / NG rows of x, go over the weights at a time.
template <int TYPE, int FMT, int NG, int AB>
__global__ __launch_bounds__(64 * kWaves) void k_few_rows(const PackedArgs a, const int kw_log2) {
  constexpr int kTok = 16 / NG;       // rows of x in a left operand
  constexpr int kRows = AB * kTok;    // ... in a pass
  constexpr int kPieces = 4 / NG;     // 16-byte pieces of x that a lane loads per chunk
  constexpr int kSlots = 4 / NG;      // rows of x per lane and left operand in the result
  extern __shared__ float red[];      // [wave][kRows][16]
  const int lane = lane_id(), n = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
  const int kw = 1 << kw_log2, kpart = wave & (kw - 1);
  const int n0 = 16 * (blockIdx.x * (kWaves >> kw_log2) + (wave >> kw_log2));
  const int total = a.T * a.k;

  int e = 0, lo = blockIdx.y * kRows, hi = total, step = gridDim.y * kRows;
  if (a.offsets) {
    if (!find_bucket(a.offsets, a.E, total, blockIdx.y, &e, &lo, &hi)) return;
    step = kRows;
  }
  const int G = a.K / a.group;
  const int64_t wrow = static_cast<int64_t>(e) * a.N + min(n0 + n, a.N - 1);
  const char* codes = reinterpret_cast<const char*>(a.codes) + wrow * (a.K / 2);
  const char* scales = static_cast<const char*>(a.scales) + wrow * G * (FMT == 0 ? 2 : 1);
  const char* biases = FMT == 0 ? reinterpret_cast<const char*>(a.biases) + wrow * G * 2 : nullptr;
  const int chunks = (a.K + kChunk - 1) / kChunk;
  const int c0 = static_cast<int>(static_cast<int64_t>(chunks) * kpart / kw);
  const int c1 = static_cast<int>(static_cast<int64_t>(chunks) * (kpart + 1) / kw);
  // this lane's row of the left operand: which row of x and which group
  const int mtok = n / NG, mg = n % NG;
  const bool mine = q / kPieces == mg;

  for (int p0 = lo; p0 < hi; p0 += step) {
    const char* x[AB];
#pragma unroll
    for (int i = 0; i < AB; ++i) {
      const int p = min(p0 + i * kTok + mtok, hi - 1);
      const int row = max(row_of(a.perm, a.x_order, a.k, total, p, a.err), 0);
      x[i] = static_cast<const char*>(a.x) + static_cast<int64_t>(row) * a.K * 2;
    }
    float acc[AB][kSlots] = {};
    for (int c = c0; c < c1; ++c) {
      const int kq = c * kChunk + 32 * q;
      const bool valid = kq < a.K;
      const int at = min(kq, a.K - 32);
      const u32x4_t w = *reinterpret_cast<const u32x4_t*>(codes + at / 2);
      const packed_t<FMT, NG> s = load_groups<FMT, NG>(scales, c * NG, G);
      packed_t<FMT, NG> b = 0;
      if constexpr (FMT == 0) b = load_groups<FMT, NG>(biases, c * NG, G);
      u32x4_t wf[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) wf[i] = codes_to_16<TYPE, FMT>(w[i]);
      const uint32_t mask = valid && mine ? ~0u : 0u;
      const uint32_t one = TYPE == kBf16 ? 0x3f803f80u : 0x3c003c00u;
      const u32x4_t ones = {one, one, one, one};
#pragma unroll
      for (int t = 0; t < AB; ++t) {
        u32x4_t xp[kPieces], xf[4];
#pragma unroll
        for (int i = 0; i < kPieces; ++i)
          xp[i] = in_code_order<FMT>(*reinterpret_cast<const u32x4_t*>(x[t] + 2 * (at + 8 * (mg + NG * i))));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (NG == 1) {
#pragma unroll
            for (int j = 0; j < 4; ++j) xf[i][j] = xp[i][j] & mask;
          }
        }
        if constexpr (NG == 2) {
          xf[0] = quad_moved<0xA0>(xp[0], mask);
          xf[1] = quad_moved<0xF5>(xp[0], mask);
          xf[2] = quad_moved<0xA0>(xp[1], mask);
          xf[3] = quad_moved<0xF5>(xp[1], mask);
        }
        if constexpr (NG == 4) {
          xf[0] = quad_moved<0x00>(xp[0], mask);
          xf[1] = quad_moved<0x55>(xp[0], mask);
          xf[2] = quad_moved<0xAA>(xp[0], mask);
          xf[3] = quad_moved<0xFF>(xp[0], mask);
        }
        f32x4_t d = {0.0f, 0.0f, 0.0f, 0.0f}, sx = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < 4; ++i) d = mma16<TYPE>(xf[i], wf[i], d);
        if constexpr (FMT == 0) {
#pragma unroll
          for (int i = 0; i < 4; ++i) sx = mma16<TYPE>(xf[i], ones, sx);
        }
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          float& r = acc[t][v / NG];
          r = fmaf(group_scale<FMT, NG>(s, v % NG), d[v], r);
          if constexpr (FMT == 0) r = fmaf(group_scale<FMT, NG>(b, v % NG), sx[v], r);
        }
      }
    }
    // the waves' parts, joined in their order
    if (p0 != lo) __syncthreads();
#pragma unroll
    for (int t = 0; t < AB; ++t)
#pragma unroll
      for (int i = 0; i < kSlots; ++i)
        red[(wave * kRows + t * kTok + q * kSlots + i) * 16 + n] = acc[t][i];
    __syncthreads();
    const int tiles = kWaves >> kw_log2;
    for (int i = threadIdx.x; i < tiles * kRows * 16; i += 64 * kWaves) {
      const int col = i & 15, r = (i >> 4) % kRows, tile = (i >> 4) / kRows;
      const int row_n = 16 * (blockIdx.x * tiles + tile) + col, p = p0 + r;
      if (row_n >= a.N || p >= hi) continue;
      float v = 0.0f;
      for (int w = 0; w < kw; ++w) v += red[((tile * kw + w) * kRows + r) * 16 + col];
      const int row = row_of(a.perm, a.out_order, a.k, total, p, a.err);
      if (row < 0) continue;
      const int64_t to = static_cast<int64_t>(row) * a.N + row_n;
      if (a.out_dtype == kF32)
        static_cast<float*>(a.out)[to] = v;
      else if (a.out_dtype == kBf16)
        static_cast<uint16_t*>(a.out)[to] = static_cast<uint16_t>(f32_to_bf16_rne(v));
      else
        static_cast<uint16_t*>(a.out)[to] = __builtin_bit_cast(uint16_t, static_cast<_Float16>(v));
    }
  }
}

template <int TYPE, int FMT, int NG, int AB>
hipError_t launch_few(const PackedArgs& a, hipStream_t s) {
  constexpr int kRows = AB * 16 / NG;
  const int n = a.T * a.k;
  const int64_t tiles = (a.N + 15) / 16;
  const int64_t y = std::min(a.offsets ? std::min(n, a.E) : (n + kRows - 1) / kRows, 65535);
  int kw_log2 = 0;
  const int chunks = (a.K + kChunk - 1) / kChunk;
  while (kw_log2 < 3 && (tiles * y << kw_log2) < 4096 && (chunks >> kw_log2) > 2) ++kw_log2;
  const int64_t gx = (tiles + (kWaves >> kw_log2) - 1) / (kWaves >> kw_log2);
  if (gx * y > max_workgroups(64 * kWaves)) return hipErrorInvalidValue;
  QSMOE_LAUNCH((k_few_rows<TYPE, FMT, NG, AB>), dim3(static_cast<unsigned>(gx), static_cast<unsigned>(y)),
               dim3(64 * kWaves), kWaves * kRows * 16 * sizeof(float), s, a, kw_log2);
  return hipGetLastError();
}

template <int TYPE, int FMT, int NG>
hipError_t pick_rows(const PackedArgs& a, hipStream_t s) {
  constexpr int kTok = 16 / NG;
  const int64_t n = static_cast<int64_t>(a.T) * a.k;
  const int64_t rows = a.offsets ? (n + a.E - 1) / a.E : n;  // of a pass, on average
  if (rows <= kTok) return launch_few<TYPE, FMT, NG, 1>(a, s);
  if (rows <= 2 * kTok) return launch_few<TYPE, FMT, NG, 2>(a, s);
  return launch_few<TYPE, FMT, NG, 4>(a, s);
}

template <int TYPE>
hipError_t pick_groups(const PackedArgs& a, hipStream_t s) {
  if (!a.biases) return pick_rows<TYPE, 1, 4>(a, s);
  if (a.group == 32) return pick_rows<TYPE, 0, 4>(a, s);
  if (a.group == 64) return pick_rows<TYPE, 0, 2>(a, s);
  return pick_rows<TYPE, 0, 1>(a, s);
}

}  // namespace

hipError_t launch_product_packed(const PackedArgs& a, hipStream_t s) {
  return a.dtype == kBf16 ? pick_groups<kBf16>(a, s) : pick_groups<kF16>(a, s);
}

}  // namespace qsmoe

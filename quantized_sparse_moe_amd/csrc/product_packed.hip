// Products of few rows with 4-bit weights, dense or grouped by expert:
//   out[p][n] = sum_k x[p][k] W[n][k],
// W affine (w = s q + b, fp16 s and b per group of 32, 64 or 128) or MXFP4 (w =
// 2^(s - 127) e2m1(q) per 32). Within a group g of a row n
//   sum_k x w = s (sum_k x q) + b (sum_k x),
// so the codes go to the matrix cores as they are, exact in bf16 and fp16, and
// scales and biases touch each group's sum only.
//
// The weights are the right operand of v_mfma_f32_16x16x32: lane (n, q), n =
// lane % 16, q = lane / 16, loads 16 bytes, the 32 codes of quarter q of row n's
// 128-code chunk, so that a wave reads 64 bytes of each of 16 rows. Four lane
// swaps turn quarter q's word i into quarter i's word q: product i then covers
// quarter i alone, 32 codes of one group, and a group's products are summed from
// zero before its scale multiplies them. Unpacking takes 36 instructions per
// chunk, 1.1 a code and lane, which the vector units do at twice the rate at
// which HBM delivers codes.
//
// k_few_rows streams a matrix past up to 16 rows of x in LDS, k_many_rows goes over
// it with tiles of 16 to 64 rows, k_small is for products that end before a stream
// has begun. k_short_rows takes contractions shorter than a chunk.
#include <algorithm>
#include <atomic>

#include "elements.hpp"
#include "kernels.hpp"
#include "product_core.hpp"

namespace qsmoe {

namespace {

constexpr int kLds = 160 * 1024;  // of a CU
constexpr int kMostWaves = 8;
constexpr int kChunk = 128, kStepChunks = 4, kStep = kStepChunks * kChunk;

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

template <int TYPE>
__device__ __forceinline__ float sum_of_8(u32x4_t x) {
  float v = 0.0f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (TYPE == kBf16)
      v += __uint_as_float(x[j] << 16) + __uint_as_float(x[j] & 0xffff0000u);
    else
      v += f16_to_f32(static_cast<uint16_t>(x[j])) + f16_to_f32(static_cast<uint16_t>(x[j] >> 16));
  }
  return v;
}

// Lane (n, q)'s word i, of quarter q, for word q of quarter i: a 4 x 4
// transposition over the wave's rows of 16 lanes, by two exchanges of rows 0 and
// 1 (2 and 3) and two of the halves.
__device__ __forceinline__ u32x4_t quarters_together(u32x4_t w) {
  const auto ab = __builtin_amdgcn_permlane16_swap(w[0], w[1], false, false);
  const auto cd = __builtin_amdgcn_permlane16_swap(w[2], w[3], false, false);
  const auto ac = __builtin_amdgcn_permlane32_swap(ab[0], cd[0], false, false);
  const auto bd = __builtin_amdgcn_permlane32_swap(ab[1], cd[1], false, false);
  return u32x4_t{ac[0], bd[0], ac[1], bd[1]};
}

// Scales, or biases, of a row's groups: fp16 (affine) or e8m0 bytes.
template <int FMT, int NG>
struct Groups {
  static constexpr int kSize = FMT == 0 ? 2 : 1;
  static constexpr int kStepBytes = kStepChunks * NG * kSize;
  static constexpr int kBlockSteps = 64 / kStepBytes;  // steps of a 64-byte block, four lanes' pieces
};

// 16 bytes of a row's group values from byte `at` on; `left`: bytes of the whole
// array from the row on. A row may start at any element, so the vector promises
// no more. What lies behind the row's end is for within_row to take out, once the
// bytes are used: here it would wait for them.
__device__ __forceinline__ u32x4_t load_piece(const char* row, int at, int64_t left) {
  u32x4_t v;
  if (at + 16 <= left) {
    __builtin_memcpy(&v, row + at, 16);
  } else {  // the array ends: each word as far back as it has to be
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t w;
      __builtin_memcpy(&w, row + min(static_cast<int64_t>(at + 4 * j), left - 4), 4);
      v[j] = w;
    }
  }
  return v;
}
__device__ __forceinline__ u32x4_t within_row(u32x4_t v, int at, int row_bytes, int64_t left) {
  if (at + 16 <= row_bytes) return v;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int exist = row_bytes - at - 4 * j;  // bytes of this word
    const int64_t back = at + 4 * j + 4 - left;
    uint32_t w = v[j];
    if (back > 0) w = back < 4 ? w >> (8 * static_cast<int>(back)) : 0u;
    v[j] = exist >= 4 ? w : exist <= 0 ? 0u : w & ((1u << (8 * exist)) - 1u);
  }
  return v;
}

template <int FMT>
__device__ __forceinline__ float group_value(const uint32_t* v, int i) {
  if constexpr (FMT == 0)
    return f16_to_f32(static_cast<uint16_t>(v[i / 2] >> (16 * (i % 2))));
  else
    return e8m0_to_f32((v[i / 4] >> (8 * (i % 4))) & 0xffu);
}

// The b-th run of up to `most` rows of one expert: its expert, first position and
// rows. Offsets are clamped to [0, n]; without them all rows are one expert's.
// Uniform over the wave: 4 experts a lane, their runs scanned. So long buckets
// take as many workgroups more as they have runs (280 tokens' top-7 of 214 experts
// of 479 x 864, the most popular with 280 rows: 167 us with a bucket's runs one
// after the other, 35 side by side).
__device__ __forceinline__ bool find_run(const int32_t* offsets, int E, int n, int b, int most, int* e, int* first,
                                         int* rows) {
  if (!offsets) {
    *e = 0;
    *first = b * most;
    *rows = min(most, n - *first);
    return *rows > 0;
  }
  const int lane = lane_id();
  int before = 0;
  for (int e0 = 0; e0 < E; e0 += 256) {
    const int i = e0 + 4 * lane;
    int o[5], runs[4], sum = 0;
#pragma unroll
    for (int v = 0; v < 5; ++v) o[v] = min(max(offsets[min(i + v, E)], 0), n);
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const uint32_t len = max(o[v + 1] - o[v], 0);  // 0 past the last expert
      runs[v] = (len + most - 1) / static_cast<uint32_t>(most);
      sum += runs[v];
    }
    const int incl = wave_scan(sum);
    const uint64_t m = __ballot(before + incl > b);
    if (m != 0) {
      const int src = __ffsll(static_cast<unsigned long long>(m)) - 1;
      int at = b - before - __builtin_amdgcn_readlane(incl - sum, src);  // run among the lane's
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int here = __builtin_amdgcn_readlane(runs[v], src);
        if (at < here) {
          *e = e0 + 4 * src + v;
          *first = __builtin_amdgcn_readlane(o[v], src) + at * most;
          *rows = min(most, __builtin_amdgcn_readlane(o[v + 1], src) - *first);
          return true;
        }
        at -= here;
      }
      return false;
    }
    before += __builtin_amdgcn_readlane(incl, 63);
  }
  return false;
}

// Words from LDS, 8 or 16 bytes at a time.
template <int WORDS>
__device__ __forceinline__ void lds_words(const char* p, uint32_t (&v)[WORDS]) {
  if constexpr (WORDS == 2) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    v[0] = u.x;
    v[1] = u.y;
  } else {
#pragma unroll
    for (int i = 0; i < WORDS; i += 4) {
      const u32x4_t u = lds16(p + 4 * i);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[i + j] = u[j];
    }
  }
}

// LDS of k_few_rows: a wave's scales (and biases) of 16 rows, 80 bytes apart,
// which no two rows' reads share a bank at; rows of x, 64 bytes apart in the banks.
constexpr int kValueRow = 80, kPad = 64;
template <int FMT>
constexpr int kValueLds = (FMT == 0 ? 2 : 1) * 16 * kValueRow;

__device__ __forceinline__ void store_value(const PackedArgs& a, int row, int n, float v) {
  const int64_t to = static_cast<int64_t>(row) * a.N + n;
  if (a.out_dtype == kF32)
    static_cast<float*>(a.out)[to] = v;
  else if (a.out_dtype == kBf16)
    static_cast<uint16_t*>(a.out)[to] = static_cast<uint16_t>(f32_to_bf16_rne(v));
  else
    static_cast<uint16_t*>(a.out)[to] = __builtin_bit_cast(uint16_t, static_cast<_Float16>(v));
}

// Row r of x in a left operand of 4 VR rows, from its row m of 16, or -1. Element
// v of lane (n, q) in the result is its row 4 q + v, which holds row 4 v + q of x:
// up to 4 rows of x need one element a lane and one multiplication by each scale
// (k_small), 8 two, 16 four (k_few_rows).
template <int VR>
__device__ __forceinline__ int x_row(int m) {
  return m % 4 < VR ? m % 4 * 4 + m / 4 : -1;
}

// How a launch is laid out: runs of up to `most` rows; 2^kw_log2 of a workgroup's
// waves share a tile's contraction, `own` steps each of every segment of `seg` steps,
// as much of x as fits in LDS.
struct FewShape {
  int32_t most, kw_log2, seg, own;
};

// A tile is 16 rows of W. A workgroup keeps its rows of x (4 VR at a time) in LDS
// and goes over its tiles with them. A wave loads the codes of its next step, of
// the next tile where one ends, before it multiplies the present one. Scales and
// biases it loads in blocks of 64 bytes a row, as wide as the codes: 16 bytes a
// step, the same for all four quarters, fetch each of their lines 8 times (129280 x
// 4096, groups of 64: 72 to 77 us so, 61 to 65 in blocks). Their lanes meet the
// multiplying ones through the wave's own part of LDS.
//
// HBM bounds it: 129280 x 4096 with one row 57 to 65 us, 4.6 to 5.2 TB/s; 64
// tokens' top-6 of 256 experts of 4096 x 4096 314 us, 5.4 TB/s of the experts that
// are expected in use; 512 tokens (12 rows a bucket, several runs where it is
// popular) 634. Loads that bypass the caches are 2 to 6 % slower. A third wave to a
// SIMD is worth the registers that it costs, but only short rows of x leave room for
// it: 3, 8 and 16 rows of 32768 x 8192 have two (the counters say so too) and take
// 42, 48 and 55 us where one row takes 35. Buckets of 17 rows and more stream their
// weights once per run of 16: about 18 rows of each of 64 experts of 4096 x 4096 212 to
// 249 us, where 570 MB of weights are needed and 970 MB read.
// WHOLE: a row's values and the steps at which a wave's blocks of them begin are
// multiples of 16 bytes, so that none of the pieces ends behind its row.
template <int TYPE, int FMT, int NG, int VR, bool WHOLE>
__global__ __launch_bounds__(64 * kMostWaves) __attribute__((amdgpu_waves_per_eu(3)))
void k_few_rows(const PackedArgs a, const FewShape f) {
  using Values = Groups<FMT, NG>;
  constexpr int kStepBytes = 2 * kStep;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int lane = lane_id(), n = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
  const int waves = blockDim.x >> 6, kw = 1 << f.kw_log2, kpart = wave & (kw - 1), sub = wave >> f.kw_log2;
  const int subs = waves >> f.kw_log2;
  const int groups = ((a.N + 15) / 16 + subs - 1) / subs;  // of tiles, one per `sub`
  const int total = a.T * a.k;

  int e, p0, rows;
  if (!find_run(a.offsets, a.E, total, blockIdx.y, f.most, &e, &p0, &rows)) return;
  const int steps = (a.K + kStep - 1) / kStep;
  const int value_bytes = a.K / a.group * Values::kSize;  // of a row
  const int64_t all_values = static_cast<int64_t>(a.E) * a.N * value_bytes;

  // this wave's steps: step i is the (i % own)-th of its share of segment i / own
  const int whole = steps / f.seg;
  const int mine = whole * f.own + min(max(steps - whole * f.seg - kpart * f.own, 0), f.own);
  auto step_of = [&](int i) { return i / f.own * f.seg + kpart * f.own + i % f.own; };
  auto w_row = [&](int group) { return static_cast<int64_t>(e) * a.N + min(16 * (group * subs + sub) + n, a.N - 1); };
  // Codes past a row's end are its last ones again, for which x is zero.
  auto load_codes = [&](int group, int i, u32x4_t (&w)[kStepChunks]) {
    const int step = step_of(i);
    const char* row = reinterpret_cast<const char*>(a.codes) + w_row(group) * (a.K / 2);
#pragma unroll
    for (int h = 0; h < kStepChunks; ++h)
      w[h] = *reinterpret_cast<const u32x4_t*>(row + min(step * kStep + h * kChunk + 32 * q, a.K - 32) / 2);
  };
  auto load_values = [&](int group, int i, u32x4_t& s, u32x4_t& b) {
    int at = step_of(i) * Values::kStepBytes + 16 * q;
    int64_t row = w_row(group) * value_bytes, left = all_values - row;
    if constexpr (WHOLE) {  // a piece past the row's end is its last one: its codes' x is zero
      at = min(at, value_bytes - 16);
      left = at + 16;
    }
    s = load_piece(static_cast<const char*>(a.scales) + row, at, left);
    if constexpr (FMT == 0) b = load_piece(reinterpret_cast<const char*>(a.biases) + row, at, left);
  };

  // LDS: the waves' blocks of scales and biases, rows 80 bytes apart; the rows of
  // x, their sums per group, the waves' parts of a tile
  char* values = lds + wave * kValueLds<FMT>;
  char* xs = lds + waves * kValueLds<FMT>;
  const int row_bytes = f.seg * kStepBytes + kPad, seg_groups = f.seg * kStepChunks * NG;
  float* sums = reinterpret_cast<float*>(xs + rows * row_bytes);
  float* red = sums + (FMT == 0 ? rows * seg_groups : 0);
  // where this lane finds its row of the left operand, and its rows' sums; the
  // operand's other rows are row 0 again, and their results are not kept
  const int from_row = x_row<VR>(n);
  const int at = (from_row >= 0 && from_row < rows ? from_row : 0) * row_bytes + 16 * q;
  int sum_at[VR];
#pragma unroll
  for (int v = 0; v < VR; ++v) sum_at[v] = min(4 * v + q, rows - 1) * seg_groups;
  // x's columns of steps seg0 .. seg_end - 1: a workgroup's threads take
  // neighbouring pieces of one row, several rows or runs of pieces in flight
  auto stage = [&](int seg0, int seg_end) {
    constexpr int kAhead = 2;
    const int pieces = (seg_end - seg0) * (kStep / 8);
    for (int r = 0, j0 = 0; j0 < pieces;) {
      u32x4_t v[kAhead];
      int to[kAhead];  // where a piece goes, -1: none
      int sum_to[kAhead];
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int j = j0 + threadIdx.x;
        to[u] = -1;
        if (j < pieces) {
          const int step = seg0 + j / (kStep / 8);
          const int k = step * kStep + j % (kStep / 8) * 8;
          const int row = max(row_of(a.perm, a.x_order, a.k, total, p0 + r, a.err), 0);
          v[u] = u32x4_t{0, 0, 0, 0};
          if (k < a.K)
            v[u] = *reinterpret_cast<const u32x4_t*>(static_cast<const char*>(a.x) +
                                                     2 * (static_cast<int64_t>(row) * a.K + k));
          to[u] = r * row_bytes + 16 * j;
          sum_to[u] = r * seg_groups + j / (16 / NG);
        }
        if (++r == rows) {
          r = 0;
          j0 += blockDim.x;
        }
      }
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (to[u] < 0) continue;  // the same for a whole wave: pieces is a multiple of 64
        *reinterpret_cast<u32x4_t*>(xs + to[u]) = in_code_order<FMT>(v[u]);
        if constexpr (FMT == 0) {
          float s = sum_of_8<TYPE>(v[u]);
#pragma unroll
          for (int o = 1; o < 16 / NG; o <<= 1) s += xchg(s, o);
          if (lane % (16 / NG) == 0) sums[sum_to[u]] = s;
        }
      }
    }
  };

  u32x4_t cur[kStepChunks], ahead[kStepChunks], next_s, next_b;
  float acc[VR];
  auto multiply = [&](int in_seg, int in_block) {
    uint32_t s[Values::kStepBytes / 4], b[Values::kStepBytes / 4];
    const char* v = values + n * kValueRow + in_block * Values::kStepBytes;
    lds_words(v, s);
    if constexpr (FMT == 0) lds_words(v + 16 * kValueRow, b);
#pragma unroll
    for (int h = 0; h < kStepChunks; ++h) {
      __builtin_amdgcn_sched_barrier(0);  // chunk by chunk, for the registers
      const u32x4_t w = quarters_together(cur[h]);
      u32x4_t wf[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) wf[i] = codes_to_16<TYPE, FMT>(w[i]);
      const char* xp = xs + at + in_seg * kStepBytes + h * 256;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        f32x4_t d = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 4 / NG * g; i < 4 / NG * (g + 1); ++i)
          d = mma16<TYPE>(lds16(xp + 64 * i), wf[i], d);
#pragma unroll
        for (int r = 0; r < VR; ++r) {
          acc[r] = fmaf(group_value<FMT>(s, h * NG + g), d[r], acc[r]);
          if constexpr (FMT == 0)
            acc[r] = fmaf(group_value<FMT>(b, h * NG + g), sums[sum_at[r] + (in_seg * kStepChunks + h) * NG + g],
                          acc[r]);
        }
      }
    }
  };

  const int first_group = blockIdx.x, turns = gridDim.x;
  int buffer = 0;
  if (mine > 0) {
    load_values(first_group, 0, next_s, next_b);
    load_codes(first_group, 0, cur);
  }
  for (int group = first_group; group < groups; group += turns) {
#pragma unroll
    for (int v = 0; v < VR; ++v) acc[v] = 0.0f;
    const int then = group + turns < groups ? group + turns : -1;
    int i = 0;
    for (int seg0 = 0; seg0 < steps; seg0 += f.seg) {
      const int seg_end = min(seg0 + f.seg, steps);
      if (f.seg < steps || group == first_group) {
        if (seg0 != 0 || group != first_group) lds_barrier();  // the segment before has been read
        stage(seg0, seg_end);
        lds_barrier();
      }
      const int share = min(mine - i, f.own);
      for (int j = 0; j < share; ++j, ++i) {
        const int in_block = j % Values::kBlockSteps;
        if (in_block == 0) {
          // a wave's LDS accesses are made in order: only the compiler is held
          __builtin_amdgcn_wave_barrier();
          char* v = values + n * kValueRow + 16 * q;
          if constexpr (!WHOLE) {
            const int from = step_of(i) * Values::kStepBytes + 16 * q;
            const int64_t left = all_values - w_row(group) * value_bytes;
            next_s = within_row(next_s, from, value_bytes, left);
            if constexpr (FMT == 0) next_b = within_row(next_b, from, value_bytes, left);
          }
          *reinterpret_cast<u32x4_t*>(v) = next_s;
          if constexpr (FMT == 0) *reinterpret_cast<u32x4_t*>(v + 16 * kValueRow) = next_b;
          __builtin_amdgcn_wave_barrier();
          const int block = j + Values::kBlockSteps < share ? i + Values::kBlockSteps : i - j + share;
          if (block < mine)
            load_values(group, block, next_s, next_b);
          else if (then >= 0)
            load_values(then, 0, next_s, next_b);
        }
        const int in_seg = kpart * f.own + j, next_group = i + 1 < mine ? group : then;
        if (next_group >= 0) {
          load_codes(next_group, i + 1 < mine ? i + 1 : 0, ahead);
          multiply(in_seg, in_block);
#pragma unroll
          for (int h = 0; h < kStepChunks; ++h) cur[h] = ahead[h];
        } else {
          multiply(in_seg, in_block);
        }
      }
    }
    if (kw == 1) {
      const int row_n = 16 * (group * subs + sub) + n;
#pragma unroll
      for (int v = 0; v < VR; ++v) {
        const int r = 4 * v + q;
        if (r >= rows || row_n >= a.N) continue;
        const int row = row_of(a.perm, a.out_order, a.k, total, p0 + r, a.err);
        if (row >= 0) store_value(a, row, row_n, acc[v]);
      }
      continue;
    }
    // the waves' parts, joined in their order; two buffers in turn, so that
    // one barrier does
    float* part = red + buffer * waves * rows * 16;
    buffer ^= 1;
#pragma unroll
    for (int v = 0; v < VR; ++v)
      if (4 * v + q < rows) part[(wave * rows + 4 * v + q) * 16 + n] = acc[v];
    lds_barrier();
    for (int i = threadIdx.x; i < subs * rows * 16; i += blockDim.x) {
      const int col = i % 16, r = i / 16 % rows, of = i / 16 / rows, row_n = 16 * (group * subs + of) + col;
      if (row_n >= a.N) continue;
      float v = 0.0f;
      for (int w = 0; w < kw; ++w) v += part[((of * kw + w) * rows + r) * 16 + col];
      const int row = row_of(a.perm, a.out_order, a.k, total, p0 + r, a.err);
      if (row >= 0) store_value(a, row, row_n, v);
    }
  }
}

// The values of a chunk's NG groups of one row, packed as they lie. The last
// chunk's may end before the chunk does: they are loaded from as far back as the
// row's G groups allow, and moved to their place when used (here the shift would
// wait for them).
template <int FMT, int NG>
using chunk_values_t =
    std::conditional_t<FMT == 1 || NG == 2, uint32_t, std::conditional_t<NG == 4, uint64_t, uint16_t>>;

template <int FMT, int NG>
__device__ __forceinline__ chunk_values_t<FMT, NG> load_chunk_values(const char* row, int c, int G) {
  chunk_values_t<FMT, NG> v;
  __builtin_memcpy(&v, row + min(c * NG, G - NG) * (FMT == 0 ? 2 : 1), sizeof(v));
  return v;
}

template <int FMT, int NG>
__device__ __forceinline__ float chunk_value(chunk_values_t<FMT, NG> v, int g) {
  if constexpr (FMT == 0)
    return f16_to_f32(static_cast<uint16_t>(v >> (16 * g)));
  else
    return e8m0_to_f32(static_cast<uint32_t>(v >> (8 * g)) & 0xffu);
}

constexpr int kManyPitch = 2 * kChunk + 16;  // bytes between two rows of x in LDS

template <int TYPE>
__device__ __forceinline__ u32x4_t ones_16() {
  constexpr uint32_t one = TYPE == kBf16 ? 0x3f803f80u : 0x3c003c00u;
  return u32x4_t{one, one, one, one};
}

// One row's codes of a chunk and their scales and biases.
template <int FMT, int NG>
struct Chunk {
  u32x4_t w;
  chunk_values_t<FMT, NG> s, b;

  __device__ __forceinline__ void settle(int c, int G) {  // chunk c's values in their places
    const int by = 8 * (FMT == 0 ? 2 : 1) * max(c * NG - (G - NG), 0);
    s = static_cast<chunk_values_t<FMT, NG>>(s >> by);
    if constexpr (FMT == 0) b = static_cast<chunk_values_t<FMT, NG>>(b >> by);
  }
};
template <int FMT, int NG>
__device__ __forceinline__ Chunk<FMT, NG> load_chunk(const char* codes, const char* scales, const char* biases, int c,
                                                     int q, int K, int G) {
  Chunk<FMT, NG> r;
  r.w = *reinterpret_cast<const u32x4_t*>(codes + min(c * kChunk + 32 * q, K - 32) / 2);
  r.s = load_chunk_values<FMT, NG>(scales, c, G);
  if constexpr (FMT == 0) r.b = load_chunk_values<FMT, NG>(biases, c, G);
  return r;
}

// More rows of x: tiles of 16 AB rows by 16 RT rows of W a wave; x is staged for
// all waves, CH chunks at a time for each of the KW waves that share a
// contraction, two buffers in turn. The sums of x come from products with ones,
// as the matrix cores have the time. Loads stand outside of branches and values
// are shifted to their places when used: with either one the other way round the
// compiler waits for all loads of a stage (64 rows of 4096 x 4096: 26 us, now 19).
// A chunk is 36 + 16 NG AB vector instructions against 4 (AB + 1) matrix products
// (1024 rows of 4096 x 4096 70 to 79 us, 0.43 to 0.49 PFLOP/s: matrix units busy 31 %
// of the time). With 17 to 64 rows neither bounds it: 64 rows of 32768 x 8192, groups
// of 128, 90 to 98 us, matrix units busy 24 %, vector instructions issued 45 %, and
// the waves wait 36 % of their time. Two waves a SIMD are all that 136 KB of LDS and
// up to 256 registers leave (AB 4, KW 4), and each stage ends in a barrier for eight
// waves. 64 rows of 4096 x 4096: 128 workgroups, half of the CUs, 19 us.
template <int TYPE, int FMT, int NG, int AB, int RT, int CH, int KW>
__global__ __launch_bounds__(64 * kMostWaves) void k_many_rows(const PackedArgs a, const int ctiles, const int run) {
  constexpr int BM = 16 * AB, kw = KW, slots = KW * CH, subs = kMostWaves / KW;
  constexpr int kPieces = (slots * AB + 1) / 2;  // of 16 bytes that a thread stages
  constexpr int chunk_bytes = BM * kManyPitch, buffer_bytes = slots * chunk_bytes;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int lane = lane_id(), n = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
  const int kpart = wave % KW, sub = wave / KW;
  const int total = a.T * a.k;
  TileAt tile;
  tile.e = 0;
  if (!find_tile<BM>(a.offsets, a.E, total, ctiles, pair_of_block(run), &tile)) return;
  const int G = a.K / a.group, chunks = (a.K + kChunk - 1) / kChunk;
  const int stages = (chunks + slots - 1) / slots;
  const int n0 = 16 * RT * (tile.ctile * subs + sub);

  const char *codes[RT], *scales[RT], *biases[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) {
    const int64_t row = static_cast<int64_t>(tile.e) * a.N + min(n0 + 16 * r + n, a.N - 1);
    codes[r] = reinterpret_cast<const char*>(a.codes) + row * (a.K / 2);
    scales[r] = static_cast<const char*>(a.scales) + row * G * (FMT == 0 ? 2 : 1);
    biases[r] = FMT == 0 ? reinterpret_cast<const char*>(a.biases) + row * G * 2 : nullptr;
  }
  auto load_w = [&](int stage, Chunk<FMT, NG> (&w)[CH][RT]) {
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int r = 0; r < RT; ++r)
        w[c][r] = load_chunk<FMT, NG>(codes[r], scales[r], biases[r],
                                      min(stage * slots + kpart * CH + c, chunks - 1), q, a.K, G);
  };

  // LDS: two buffers of `slots` chunks of BM rows; in the end the waves' parts
  const char* from[kPieces];
  int left[kPieces];  // columns of x from there on
#pragma unroll
  for (int u = 0; u < kPieces; ++u) {
    const int id = threadIdx.x + 64 * kMostWaves * u, slot = id / (16 * BM), row = id / 16 % BM, j = id % 16;
    const int p = tile.first + min(row, tile.rows - 1);
    const int at = max(row_of(a.perm, a.x_order, a.k, total, p, a.err), 0);
    left[u] = a.K - slot * kChunk - 8 * j;
    from[u] = static_cast<const char*>(a.x) + 2 * (static_cast<int64_t>(at + 1) * a.K - left[u]);
  }
  // Without branches around the loads, so that the waits can count them: pieces
  // past a row's end are read at its last columns and written as zeros.
  u32x4_t xv[kPieces];
  auto load_x = [&](int stage) {
    const int k = stage * slots * kChunk;
#pragma unroll
    for (int u = 0; u < kPieces; ++u)
      xv[u] = *reinterpret_cast<const u32x4_t*>(from[u] + 2 * min(k, left[u] - 8));
  };
  auto write_x = [&](int stage, int buffer) {
    const int k = stage * slots * kChunk;
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const int id = threadIdx.x + 64 * kMostWaves * u, slot = id / (16 * BM), row = id / 16 % BM, j = id % 16;
      const u32x4_t v = k < left[u] ? xv[u] : u32x4_t{0, 0, 0, 0};
      if (slot < slots)  // the same for a whole wave
        *reinterpret_cast<u32x4_t*>(lds + buffer * buffer_bytes + slot * chunk_bytes + row * kManyPitch + 16 * j) =
            in_code_order<FMT>(v);
    }
  };

  f32x4_t acc[RT][AB] = {};
  auto multiply = [&](const char* x, int c, Chunk<FMT, NG> (&w)[RT]) {
    // in this order: interleaved with the next chunk's, more values would be live
    // than there are registers
    __builtin_amdgcn_sched_barrier(0);
    const char* xp = x + n * kManyPitch + 16 * q;
#pragma unroll
    for (int r = 0; r < RT; ++r) w[r].settle(c, G);
    u32x4_t wf[RT][4];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      const u32x4_t together = quarters_together(w[r].w);
#pragma unroll
      for (int i = 0; i < 4; ++i) wf[r][i] = codes_to_16<TYPE, FMT>(together[i]);
    }
#pragma unroll
    for (int t = 0; t < AB; ++t) {
      if (t > 0) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        f32x4_t d[RT], sx = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int r = 0; r < RT; ++r) d[r] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 4 / NG * g; i < 4 / NG * (g + 1); ++i) {
          const u32x4_t xf = lds16(xp + 16 * t * kManyPitch + 64 * i);
#pragma unroll
          for (int r = 0; r < RT; ++r) d[r] = mma16<TYPE>(xf, wf[r][i], d[r]);
          if constexpr (FMT == 0) sx = mma16<TYPE>(xf, ones_16<TYPE>(), sx);
        }
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            acc[r][t][v] = fmaf(chunk_value<FMT, NG>(w[r].s, g), d[r][v], acc[r][t][v]);
            if constexpr (FMT == 0) acc[r][t][v] = fmaf(chunk_value<FMT, NG>(w[r].b, g), sx[v], acc[r][t][v]);
          }
      }
    }
  };

  Chunk<FMT, NG> w[2][CH][RT];
  load_x(0);
  load_w(0, w[0]);
  write_x(0, 0);
  load_x(1);
  load_w(1, w[1]);
  lds_barrier();
  for (int t0 = 0; t0 < stages; t0 += 2) {
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      // a stage past the last one multiplies zeros by the last chunk's codes
      const int t = t0 + b;
      write_x(t + 1, b ^ 1);
      load_x(t + 2);
#pragma unroll
      for (int c = 0; c < CH; ++c)
        multiply(lds + b * buffer_bytes + (kpart * CH + c) * chunk_bytes,
                 min(t * slots + kpart * CH + c, chunks - 1), w[b][c]);
      __builtin_amdgcn_sched_barrier(0);
      load_w(t + 2, w[b]);
      lds_barrier();
    }
  }
  if (kw == 1) {
#pragma unroll
    for (int t = 0; t < AB; ++t)
#pragma unroll
      for (int v = 0; v < 4; ++v) {
        const int r = 16 * t + 4 * q + v;
        if (r >= tile.rows) continue;
        const int row = row_of(a.perm, a.out_order, a.k, total, tile.first + r, a.err);
        if (row < 0) continue;
#pragma unroll
        for (int i = 0; i < RT; ++i)
          if (n0 + 16 * i + n < a.N) store_value(a, row, n0 + 16 * i + n, acc[i][t][v]);
      }
    return;
  }
  // the waves' parts, joined in their order
  float* red = reinterpret_cast<float*>(lds);  // [wave][BM][16 RT]
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int t = 0; t < AB; ++t)
#pragma unroll
      for (int v = 0; v < 4; ++v) red[((wave * BM + 16 * t + 4 * q + v) * RT + i) * 16 + n] = acc[i][t][v];
  lds_barrier();
  for (int i = threadIdx.x; i < subs * tile.rows * 16 * RT; i += 64 * kMostWaves) {
    const int col = i % (16 * RT), r = i / (16 * RT) % tile.rows, of = i / (16 * RT) / tile.rows;
    const int row_n = 16 * RT * (tile.ctile * subs + of) + col;
    if (row_n >= a.N) continue;
    float v = 0.0f;
    for (int j = 0; j < kw; ++j) v += red[((of * kw + j) * BM + r) * 16 * RT + col];
    const int row = row_of(a.perm, a.out_order, a.k, total, tile.first + r, a.err);
    if (row >= 0) store_value(a, row, row_n, v);
  }
}

// Up to 4 rows of x and few tiles, which latency bounds: a tile a workgroup, its 8
// waves share the contraction, and each loads all that it needs of 4 chunks
// together, x straight into the left operand's layout. The one barrier is in front
// of joining parts. One row of 4096 x 4096: 7.5 us between calls in a graph, 2 of
// them an empty kernel's.
template <int TYPE, int FMT, int NG>
__global__ __launch_bounds__(64 * kMostWaves) void k_small(const PackedArgs a) {
  constexpr int kRows = 4;
  __shared__ float red[kMostWaves][kRows][16];
  const int lane = lane_id(), n = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
  const int total = a.T * a.k, n0 = 16 * blockIdx.x;
  int e, p0, rows;
  if (!find_run(a.offsets, a.E, total, blockIdx.y, kRows, &e, &p0, &rows)) return;
  const int G = a.K / a.group, chunks = (a.K + kChunk - 1) / kChunk;
  const int64_t w_row = static_cast<int64_t>(e) * a.N + min(n0 + n, a.N - 1);
  const char* codes = reinterpret_cast<const char*>(a.codes) + w_row * (a.K / 2);
  const char* scales = static_cast<const char*>(a.scales) + w_row * G * (FMT == 0 ? 2 : 1);
  const char* biases = FMT == 0 ? reinterpret_cast<const char*>(a.biases) + w_row * G * 2 : nullptr;
  // a share of neighbouring chunks for each wave, four at a time
  constexpr int kTogether = 4;
  const int share = (chunks + kMostWaves - 1) / kMostWaves;
  const int c0 = min(wave * share, chunks), c1 = min(c0 + share, chunks);
  const int mine = x_row<1>(n);
  const int p = p0 + (mine >= 0 && mine < rows ? mine : 0);
  const char* x = static_cast<const char*>(a.x) +
                  2 * static_cast<int64_t>(max(row_of(a.perm, a.x_order, a.k, total, p, a.err), 0)) * a.K;
  float acc = 0.0f;
  for (int c = c0; c < c1; c += kTogether) {
    Chunk<FMT, NG> w[kTogether];
    u32x4_t xv[kTogether][4];
#pragma unroll
    for (int u = 0; u < kTogether; ++u) {
      const int at = min(c + u, c1 - 1);
      w[u] = load_chunk<FMT, NG>(codes, scales, biases, at, q, a.K, G);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = at * kChunk + 32 * i + 8 * q;
        xv[u][i] = *reinterpret_cast<const u32x4_t*>(x + 2 * min(k, a.K - 8));
      }
    }
#pragma unroll
    for (int u = 0; u < kTogether; ++u) {
      w[u].settle(min(c + u, c1 - 1), G);
      const u32x4_t together = quarters_together(w[u].w);
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        f32x4_t d = {0.0f, 0.0f, 0.0f, 0.0f}, sx = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 4 / NG * g; i < 4 / NG * (g + 1); ++i) {
          // pieces past the row's end, and of a chunk taken twice, count as zeros
          const bool there = (c + u) * kChunk + 32 * i + 8 * q < a.K && c + u < c1;
          const u32x4_t xf = in_code_order<FMT>(there ? xv[u][i] : u32x4_t{0, 0, 0, 0});
          d = mma16<TYPE>(xf, codes_to_16<TYPE, FMT>(together[i]), d);
          if constexpr (FMT == 0) sx = mma16<TYPE>(xf, ones_16<TYPE>(), sx);
        }
        acc = fmaf(chunk_value<FMT, NG>(w[u].s, g), d[0], acc);
        if constexpr (FMT == 0) acc = fmaf(chunk_value<FMT, NG>(w[u].b, g), sx[0], acc);
      }
    }
  }
  red[wave][q][n] = acc;
  lds_barrier();
  for (int i = threadIdx.x; i < rows * 16; i += 64 * kMostWaves) {
    const int col = i % 16, r = i / 16;
    if (n0 + col >= a.N) continue;
    float v = 0.0f;
#pragma unroll
    for (int j = 0; j < kMostWaves; ++j) v += red[j][r][col];
    const int row = row_of(a.perm, a.out_order, a.k, total, p0 + r, a.err);
    if (row >= 0) store_value(a, row, n0 + col, v);
  }
}

// Contractions shorter than a chunk: a thread per result, which reads its row of W by
// itself and computes without matrix products. One row of 129280 x 64 4.7 us, 64 rows
// of 4096 x 64 7, 512 of 4096 x 96 43 (9.4 TFLOP/s).
template <int TYPE, int FMT>
__global__ __launch_bounds__(256) void k_short_rows(const PackedArgs a) {
  const int n = blockIdx.x * 256 + threadIdx.x, total = a.T * a.k, G = a.K / a.group;
  for (int p = blockIdx.y; p < total; p += gridDim.y) {
    int e = a.offsets ? -1 : 0;
    for (int e0 = 0; e < 0 && e0 < a.E; e0 += kWave) {
      const int i = e0 + lane_id();
      const uint64_t m = __ballot(i < a.E && a.offsets[i] <= p && p < a.offsets[i + 1]);
      if (m != 0) e = e0 + __ffsll(static_cast<unsigned long long>(m)) - 1;
    }
    if (e < 0 || n >= a.N) continue;
    const int64_t w = static_cast<int64_t>(e) * a.N + n;
    const int row = max(row_of(a.perm, a.x_order, a.k, total, p, a.err), 0);
    const uint4* x =
        reinterpret_cast<const uint4*>(static_cast<const char*>(a.x) + 2 * static_cast<int64_t>(row) * a.K);
    float acc = 0.0f;
    for (int g = 0; g < G; ++g) {
      float dot = 0.0f, sum = 0.0f;
      for (int i = g * a.group / 8; i < (g + 1) * a.group / 8; ++i) {
        const uint32_t c = a.codes[w * (a.K / 8) + i];
        const uint4 v = x[i];
        const uint32_t words[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const uint32_t bits = words[j / 2] >> (16 * (j % 2)) & 0xffffu, q = c >> (4 * j) & 15u;
          const float f = TYPE == kBf16 ? bf16_to_f32(bits) : f16_to_f32(static_cast<uint16_t>(bits));
          float value = static_cast<float>(q);
          if constexpr (FMT != 0) {
            const uint32_t m = q & 7u;
            value = m < 5 ? 0.5f * m : m < 6 ? 3.0f : m < 7 ? 4.0f : 6.0f;
            if (q & 8u) value = -value;
          }
          dot = fmaf(f, value, dot);
          sum += f;
        }
      }
      if constexpr (FMT == 0)
        acc = fmaf(f16_to_f32(a.biases[w * G + g]), sum,
                   fmaf(f16_to_f32(static_cast<const uint16_t*>(a.scales)[w * G + g]), dot, acc));
      else
        acc = fmaf(e8m0_to_f32(static_cast<const uint8_t*>(a.scales)[w * G + g]), dot, acc);
    }
    const int to = row_of(a.perm, a.out_order, a.k, total, p, a.err);
    if (to >= 0) store_value(a, to, n, acc);
  }
}

// Which kernel, measured on both sides (bf16, groups of 64, weights of 4096 x 4096
// unless said):
//  - Buckets of more than 20 rows on average go to k_many_rows. k_few_rows and
//    k_many_rows: 18 rows of each of 64 experts (groups of 128) 212 and 251 us, 24
//    rows 270 and 252; 18 rows of 16 experts of 2048 x 2048 33 and 39 us, 32 rows 51
//    and 42; 512 tokens' top-6 of 256 experts (12 rows) 634 and 1200. Dense products
//    take the same border, though 17 to 20 of their rows are two runs, which stream
//    the matrix twice: 18 rows of 16384 x 2048 (groups of 32) 19.4 us, 24 rows 15.5;
//    of 32768 x 4096 38 and 42.
//  - Up to 512 tiles of 16 rows of W, all buckets together, are no stream: up to 4
//    rows k_small (7.5 us; k_few_rows 8.2, k_many_rows 13), from 5 on k_many_rows
//    (13 rows of 2053 x 4000, groups of 32: 8.1 us; with all of x in registers as in
//    k_small 9.0). Six experts with a row each (1536 tiles) 29 us with k_small and
//    15 with k_few_rows.
//  - Tiles of k_many_rows are as wide as leaves 192 workgroups (64 rows of 32768 x
//    8192, groups of 128: 118 us when it was chosen, 143 with 400, 207 with 96; 90 to
//    98 now).
constexpr int64_t kFewRows = 20, kSmallTiles = 512, kEnoughGroups = 192;

// The kernel steps on by grid.y: no more of it than a grid's threads leave room for.
template <int TYPE, int FMT>
hipError_t launch_short(const PackedArgs& a, hipStream_t s) {
  const int columns = (a.N + 255) / 256;
  const int64_t most_rows = std::min<int64_t>(65535, max_workgroups(256) / columns);
  const dim3 grid(columns, static_cast<unsigned>(std::min<int64_t>(int64_t{a.T} * a.k, most_rows)));
  QSMOE_LAUNCH((k_short_rows<TYPE, FMT>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

// Runs of up to `most` rows that the buckets can have together (find_run), each of a
// row at least.
int64_t most_runs(const PackedArgs& a, int most) {
  const int64_t n = static_cast<int64_t>(a.T) * a.k;
  return a.offsets ? std::min(n, std::min<int64_t>(n, a.E) + n / most) : (n + most - 1) / most;
}
constexpr int64_t kMostY = 65535;

// More than the default 64 KiB of dynamic LDS, allowed once for each kernel and
// device.
template <auto KERNEL>
hipError_t allow_lds() {
  static std::atomic<uint64_t> allowed{0};
  int device = 0;
  if (const hipError_t e = hipGetDevice(&device); e != hipSuccess) return e;
  const uint64_t bit = device < 64 ? uint64_t{1} << device : 0;
  if (allowed.load(std::memory_order_relaxed) & bit) return hipSuccess;
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(KERNEL),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
  if (e == hipSuccess) allowed.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

template <int TYPE, int FMT, int NG, int VR>
hipError_t launch_few(const PackedArgs& a, hipStream_t s) {
  const int n = a.T * a.k, steps = (a.K + kStep - 1) / kStep;
  // A token's experts are different ones as a rule, so a run need not hold more rows
  // than there are tokens (or rows in the average bucket). The less of x there is in
  // LDS, the more workgroups share a CU: top-6 experts of 4096 x 4096, 1 token 14.6
  // us, 16.7 with runs of 8; 2 tokens 23 and 30, 4 tokens 46 and 52.
  const int buckets = a.offsets ? std::min(n, a.E) : 1;
  const int most = std::min(4 * VR, std::max(a.T, (n + buckets - 1) / buckets)), rows = std::min(most, n);
  const int64_t tiles = (a.N + 15) / 16;
  const int64_t y = most_runs(a, most);
  const int step_bytes = rows * (2 * kStep + (FMT == 0 ? kStepChunks * NG * 4 : 0));
  // LDS beside the steps of x
  auto fixed = [&](int waves, int kw) {
    return rows * kPad + waves * kValueLds<FMT> + (kw == 1 ? 0 : 2 * waves * rows * 16 * 4);
  };
  // Small workgroups, three to a CU, where x and the parts leave them the room
  // (a token's six experts of 4096 x 4096: 14.6 us; 18 with one of 8 waves; four to
  // a CU are no faster).
  const int waves = fixed(4, 4) + steps * step_bytes <= kLds / 3 ? 4 : kMostWaves, per_cu = waves == 4 ? 3 : 1;
  // As few waves to a contraction as still give every wave a tile.
  int kw_log2 = 0;
  while ((2 << kw_log2) <= waves && (2 << kw_log2) <= steps && (tiles * y << kw_log2) < 256 * per_cu * waves &&
         fixed(waves, 2) + (step_bytes << (kw_log2 + 1)) <= kLds)
    ++kw_log2;
  const int kw = 1 << kw_log2, subs = waves >> kw_log2;
  const int fit = (kLds / per_cu - fixed(waves, kw)) / step_bytes;
  const int own = fit >= (steps + kw - 1) / kw * kw ? (steps + kw - 1) / kw : fit / kw, seg = own * kw;
  const int64_t groups = (tiles + subs - 1) / subs;
  // As many workgroups as run at once, each with as many groups of tiles; four
  // times as many where buckets may be empty or long.
  const int64_t at_once = 256 * per_cu * (y > 8 ? 4 : 1), turns = (groups * y + at_once - 1) / at_once;
  const int64_t gx = (groups + turns - 1) / turns;
  if (y > kMostY || gx * y > max_workgroups(64 * kMostWaves)) return hipErrorInvalidValue;
  const size_t lds = fixed(waves, kw) + static_cast<size_t>(seg) * step_bytes;
  auto launch = [&](hipError_t allowed, auto kernel) {
    if (allowed != hipSuccess) return allowed;
    QSMOE_LAUNCH(kernel, dim3(static_cast<unsigned>(gx), static_cast<unsigned>(y)), dim3(64 * waves), lds, s, a,
                 FewShape{most, kw_log2, seg, own});
    return hipGetLastError();
  };
  // pieces start at multiples of 16 bytes too: of the steps of 8 bytes at even ones
  const bool even = Groups<FMT, NG>::kStepBytes >= 16 || own % 2 == 0 || (kw == 1 && seg >= steps);
  if (a.K / a.group * Groups<FMT, NG>::kSize % 16 == 0 && even)
    return launch(allow_lds<k_few_rows<TYPE, FMT, NG, VR, true>>(), k_few_rows<TYPE, FMT, NG, VR, true>);
  return launch(allow_lds<k_few_rows<TYPE, FMT, NG, VR, false>>(), k_few_rows<TYPE, FMT, NG, VR, false>);
}

template <int TYPE, int FMT, int NG>
hipError_t launch_small(const PackedArgs& a, hipStream_t s) {
  const int64_t tiles = (a.N + 15) / 16, y = most_runs(a, 4);
  if (y > kMostY || tiles * y > max_workgroups(64 * kMostWaves)) return hipErrorInvalidValue;
  QSMOE_LAUNCH((k_small<TYPE, FMT, NG>), dim3(static_cast<unsigned>(tiles), static_cast<unsigned>(y)),
               dim3(64 * kMostWaves), 0, s, a);
  return hipGetLastError();
}

template <int TYPE, int FMT, int NG, int AB, int RT, int CH, int KW>
hipError_t launch_many(const PackedArgs& a, hipStream_t s) {
  constexpr int BM = 16 * AB, columns = 16 * RT * kMostWaves / KW;
  const int64_t n = static_cast<int64_t>(a.T) * a.k;
  const int ctiles = (a.N + columns - 1) / columns;
  const int64_t rtiles = a.offsets ? std::min<int64_t>(n, a.E) + n / BM : (n + BM - 1) / BM;
  constexpr int run = 8;  // neighbouring tiles on one XCD
  const int64_t pairs = (rtiles * ctiles + 8 * run - 1) / (8 * run) * (8 * run);
  if (pairs > max_workgroups(64 * kMostWaves)) return hipErrorInvalidValue;
  constexpr size_t lds = std::max<size_t>(2 * KW * CH * BM * kManyPitch, KW == 1 ? 0 : kMostWaves * BM * 16 * RT * 4);
  static_assert(lds <= kLds, "LDS of a CU");
  if (const hipError_t e = allow_lds<k_many_rows<TYPE, FMT, NG, AB, RT, CH, KW>>(); e != hipSuccess) return e;
  QSMOE_LAUNCH((k_many_rows<TYPE, FMT, NG, AB, RT, CH, KW>), dim3(static_cast<unsigned>(pairs)),
               dim3(64 * kMostWaves), lds, s, a, ctiles, run);
  return hipGetLastError();
}

// The widest tiles and the least sharing of a contraction that still give most
// CUs a workgroup.
template <int TYPE, int FMT, int NG, int AB>
hipError_t pick_many(const PackedArgs& a, int64_t rtiles, hipStream_t s) {
  // Tiles a wave and chunks a stage: what registers hold, but for groups of 64 with
  // AB 4 and KW 4, which take all 256 and spill 7.
  constexpr int kMost = AB == 4 && NG == 4 ? 1 : 2, CH = AB == 1 ? 2 : 1;
  auto enough = [&](int columns) { return rtiles * ((a.N + columns - 1) / columns) >= kEnoughGroups; };
  if (enough(128 * kMost)) return launch_many<TYPE, FMT, NG, AB, kMost, CH, 1>(a, s);
  if (enough(32 * kMost)) return launch_many<TYPE, FMT, NG, AB, kMost, CH, 4>(a, s);
  return launch_many<TYPE, FMT, NG, AB, 1, 1, AB == 4 ? 4 : 8>(a, s);
}

template <int TYPE, int FMT, int NG>
hipError_t pick_rows(const PackedArgs& a, hipStream_t s) {
  const int64_t n = static_cast<int64_t>(a.T) * a.k, tiles = (a.N + 15) / 16;
  // rows of a bucket: on average over all experts, and of the longer ones, roughly
  const int64_t buckets = a.offsets ? std::min<int64_t>(n, a.E) : 1, average = (n + buckets - 1) / buckets;
  const int64_t rows = a.offsets ? std::min(n, 2 * n / a.E + 2) : n;
  if (average <= kFewRows && tiles * buckets > kSmallTiles)
    return rows <= 8 ? launch_few<TYPE, FMT, NG, 2>(a, s) : launch_few<TYPE, FMT, NG, 4>(a, s);
  if (rows <= 4) return launch_small<TYPE, FMT, NG>(a, s);
  if (average <= 16) return pick_many<TYPE, FMT, NG, 1>(a, buckets, s);
  if (average <= 32) return pick_many<TYPE, FMT, NG, 2>(a, buckets * ((average + 31) / 32), s);
  return pick_many<TYPE, FMT, NG, 4>(a, buckets * ((average + 63) / 64), s);
}

template <int TYPE>
hipError_t pick_groups(const PackedArgs& a, hipStream_t s) {
  if (a.K < kChunk) return a.biases ? launch_short<TYPE, 0>(a, s) : launch_short<TYPE, 1>(a, s);
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

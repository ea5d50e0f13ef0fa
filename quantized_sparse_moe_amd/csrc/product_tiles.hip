// Matrix-core products grouped by expert:
//   out[p][c] = sum_q rows[p][q] * weights[e(p)][c][q]   (or [q][c])
// over bf16, fp16 and block-scaled E4M3, and the gradient in the weights.
//
// Tiles. A workgroup computes BM rows x BN columns of one expert; its WM x WN
// waves each BM / WM rows x 64 columns as 16 x 16 matrix-core tiles with the
// weights as the first operand, so a lane holds 4 consecutive columns of one
// row. The contraction runs in steps of 128 bytes (64 16-bit or 128 FP8
// inputs: one scale block) through S stages of LDS filled by direct
// global -> LDS loads, S - 1 steps ahead.
//
// LDS. An operand stored with the contraction contiguous keeps 128 bytes per
// row; its 16-byte pieces are exchanged within the row by an XOR with the row
// number (applied to the source address, since a direct load writes LDS in
// lane order), which spreads the 16 rows of a fragment over the banks. The
// weights' fragment t takes rows 16 (j / 4) + 4 t + j % 4 for j = 0..15, which
// leaves each lane 16 consecutive output columns over the 4 fragments. An
// operand stored across the contraction keeps 64 contraction rows of BM or BN
// values and is read with the transposing LDS read.
#include <algorithm>
#include <type_traits>

#include "product_core.hpp"

namespace qsmoe {

namespace {

constexpr int kStepBytes = 128;

__device__ __forceinline__ int swz_r(int row) { return row & 7; }
__device__ __forceinline__ int swz_c(int n) { return (n & 3) | (((n >> 4) & 1) << 2); }
// contraction-major: XOR of the 16-byte piece index, even values
__device__ __forceinline__ int swz_q(int q) { return ((q & 3) | (((q >> 3) & 1) << 2)) << 1; }

constexpr int kE4m3Wide = 4;  // E4M3 multiplied as bf16 (fp32 outputs)

template <int TYPE, int BM, int BN, int WM, int WN, int S, bool CT>
__global__ __launch_bounds__(WM* WN * 64) void k_tile_product(ProductArgs a, int run) {
  constexpr bool FP8 = TYPE == kTypeE4m3 || TYPE == kE4m3Wide;
  constexpr int ESIZE = FP8 ? 1 : 2;
  constexpr int NT = WM * WN * 64;
  constexpr int TR = BM / WM / 16;   // row fragments of a wave
  constexpr int TC = 4;              // column fragments
  constexpr int NR = BM * 8 / NT, NC = BN * 8 / NT;
  constexpr int SCALES = FP8 ? WM * WN * 256 : 0;
  constexpr int STAGE = (BM + BN) * kStepBytes + SCALES;
  constexpr int LOADS = NR + NC + (FP8 ? 1 : 0);
  static_assert(BN == WN * 64 && NR >= 1 && NC >= 1 && NT % 256 == 0, "tile shape");
  static_assert(!(FP8 && CT), "FP8 weights have the contraction contiguous");
  __shared__ __attribute__((aligned(16))) char smem[S * STAGE];

  const int n = a.T * a.k;
  const int ctiles = (a.C + BN - 1) / BN;
  TileAt t;
  if (!find_tile<BM>(a.offsets, a.E, n, ctiles, pair_of_block(run), &t)) return;
  const int tid = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int g = lane >> 4, j = lane & 15;
  const int c0 = t.ctile * BN;
  const int qbytes = a.Q * ESIZE;  // < 2^21
  const int steps = (qbytes + kStepBytes - 1) / kStepBytes;
  const int full = qbytes / kStepBytes;
  const int qb = (a.Q + 127) / 128;

  // sources of this thread's 16-byte pieces
  const int rpiece = ((tid & 7) ^ swz_r(tid >> 3)) * 16;
  const char* rp[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int p = t.first + min(i * (NT / 8) + (tid >> 3), t.rows - 1);
    const int row = max(row_of(a.perm, a.r_order, a.k, n, p, a.err), 0);
    rp[i] = static_cast<const char*>(a.r) + static_cast<int64_t>(row) * qbytes + rpiece;
  }
  const char* cbase = static_cast<const char*>(a.c) + static_cast<int64_t>(t.e) * a.C * qbytes;
  constexpr int CPR = BN / 8;  // pieces of a contraction row (CT)
  const int cpiece = ((tid & 7) ^ swz_c(tid >> 3)) * 16;
  uint32_t co[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    if constexpr (CT) {
      const int q = i * (NT / CPR) + tid / CPR;
      const int col = ((tid % CPR) ^ swz_q(q)) * 8;
      co[i] = static_cast<uint32_t>(q) * (a.C * 2) + (c0 + col < a.C ? col * 2 : 0);
    } else {
      co[i] = static_cast<uint32_t>(min(i * (NT / 8) + (tid >> 3), a.C - 1 - c0)) * qbytes + cpiece;
    }
  }
  cbase += CT ? static_cast<int64_t>(c0) * 2 : static_cast<int64_t>(c0) * qbytes;
  const int64_t cstep = CT ? static_cast<int64_t>(64) * a.C * 2 : kStepBytes;

  const float* sp = nullptr;
  const float* csc = nullptr;
  if constexpr (FP8) {
    const int p = t.first + min(tid % BM, t.rows - 1);
    const int row = max(row_of(a.perm, a.r_order, a.k, n, p, nullptr), 0);
    sp = a.r_scales + static_cast<int64_t>(row) * qb;
    csc = a.c_scales +
          (static_cast<int64_t>(t.e) * ((a.C + 127) / 128) + min((c0 + wn * 64) / 128, (a.C - 1) / 128)) * qb;
  }

  auto issue = [&](int kb) {
    char* st = smem + (kb % S) * STAGE;
    char* sr = st + wave * 1024;
    char* sc = sr + BM * kStepBytes;
    const char* cb = cbase + kb * cstep;
    if (kb < full) {
#pragma unroll
      for (int i = 0; i < NR; ++i) load_lds16(rp[i] + kb * kStepBytes, sr + i * NT * 16);
#pragma unroll
      for (int i = 0; i < NC; ++i) load_lds16(cb + co[i], sc + i * NT * 16);
    } else {  // the last step of a ragged contraction: zeros behind its end
      const u32x4_t zero = {0, 0, 0, 0};
      const int rest = qbytes - kb * kStepBytes;
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        if (rpiece < rest)
          load_lds16(rp[i] + kb * kStepBytes, sr + i * NT * 16);
        else
          *reinterpret_cast<u32x4_t*>(sr + i * NT * 16 + lane * 16) = zero;
      }
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        if (CT ? (i * (NT / CPR) + tid / CPR) * 2 < rest : cpiece < rest)
          load_lds16(cb + co[i], sc + i * NT * 16);
        else
          *reinterpret_cast<u32x4_t*>(sc + i * NT * 16 + lane * 16) = zero;
      }
    }
    if constexpr (FP8) load_lds4(sp + kb, st + (BM + BN) * kStepBytes + wave * 256);
  };

  f32x4_t acc[TR][TC];
#pragma unroll
  for (int i = 0; i < TR; ++i)
#pragma unroll
    for (int q = 0; q < TC; ++q) acc[i][q] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  // fragment addresses within a stage
  int ra[2], ca[TC];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int piece = FP8 ? 2 * g + h : 4 * h + g;
    ra[h] = (wm * TR * 16 + j) * kStepBytes + (piece ^ swz_r(j)) * 16;
    const int cn = 16 * (j >> 2) + (j & 3);
    if constexpr (!CT) ca[h] = BM * kStepBytes + (wn * 64 + cn) * kStepBytes + (piece ^ swz_c(cn)) * 16;
  }
  if constexpr (CT) {
#pragma unroll
    for (int q = 0; q < TC; ++q)
      ca[q] = BM * kStepBytes + (8 * g + (j >> 2)) * BN * 2 +
              (((wn * 64 + 16 * q) / 8 + ((j & 3) >> 1)) ^ swz_q(8 * g + (j >> 2))) * 16 + (j & 1) * 8;
  }

  float sbs = 0.0f;  // the weights' scales of 64 steps, one per lane
  auto compute = [&](int kb) {
    const char* st = smem + (kb % S) * STAGE;
    if constexpr (FP8) {
      if ((kb & 63) == 0) {
        sbs = csc[min(kb + lane, qb - 1)];
        asm volatile("" ::"v"(sbs));  // wait for it here, not in every step
      }
      const float sb = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(sbs), kb & 63));
      i32x8_t cf[TC];
#pragma unroll
      for (int q = 0; q < TC; ++q) {
        u32x4_t lo = lds16(st + ca[0] + q * 512), hi = lds16(st + ca[1] + q * 512);
        cf[q] = __builtin_bit_cast(i32x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
      }
      const float* ss = reinterpret_cast<const float*>(st + (BM + BN) * kStepBytes) + wm * TR * 16 + j;
#pragma unroll
      for (int i = 0; i < TR; ++i) {
        u32x4_t lo = lds16(st + ra[0] + i * 2048), hi = lds16(st + ra[1] + i * 2048);
        const i32x8_t rf = __builtin_bit_cast(i32x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
        const float s = ss[i * 16] * sb;
        u32x4_t rw[4];
        if constexpr (TYPE == kE4m3Wide) {
#pragma unroll
          for (int v = 0; v < 4; ++v) rw[v] = e4m3_to_bf16x8(rf[2 * v], rf[2 * v + 1]);
        }
#pragma unroll
        for (int q = 0; q < TC; ++q) {
          f32x4_t part = {0.0f, 0.0f, 0.0f, 0.0f};
          if constexpr (TYPE == kE4m3Wide) {
#pragma unroll
            for (int v = 0; v < 4; ++v)
              part = mma16<0>(e4m3_to_bf16x8(cf[q][2 * v], cf[q][2 * v + 1]), rw[v], part);
          } else {
            part = mma_fp8(cf[q], rf);
          }
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[i][q][v] = fmaf(part[v], s, acc[i][q][v]);
        }
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        u32x4_t cf[TC];
        if constexpr (CT) {
          int at[TC];
#pragma unroll
          for (int q = 0; q < TC; ++q) at[q] = lds_address(st) + ca[q];
          if (h == 0)
            lds_tr_x4<0, 8 * BN>(at, cf);
          else
            lds_tr_x4<64 * BN, 72 * BN>(at, cf);
        } else {
#pragma unroll
          for (int q = 0; q < TC; ++q) cf[q] = lds16(st + ca[h] + q * 512);
        }
#pragma unroll
        for (int i = 0; i < TR; ++i) {
          const u32x4_t rf = lds16(st + ra[h] + i * 2048);
#pragma unroll
          for (int q = 0; q < TC; ++q) acc[i][q] = mma16<TYPE>(cf[q], rf, acc[i][q]);
        }
      }
    }
  };

#pragma unroll
  for (int s = 0; s < S - 1; ++s)
    if (s < steps) issue(s);
  for (int kb = 0; kb < steps; ++kb) {
    // step kb has landed: the S - 2 steps behind it may be in flight, counted
    // only if each issued its full number of loads
    if (S > 2 && kb + S - 2 < full)
      barrier_keep<(S - 2) * LOADS>();
    else
      barrier_keep<0>();
    if (kb + S - 1 < steps) issue(kb + S - 1);
    compute(kb);
  }

  const int osize = a.out_type == 1 ? 4 : 2;
#pragma unroll
  for (int i = 0; i < TR; ++i) {
    const int r = wm * TR * 16 + 16 * i + j;
    if (r >= t.rows) continue;
    const int row = row_of(a.perm, a.out_order, a.k, n, t.first + r, a.err);
    if (row < 0) continue;
    char* o = static_cast<char*>(a.out) + static_cast<int64_t>(row) * a.C * osize;
    if constexpr (CT) {
#pragma unroll
      for (int q = 0; q < TC; ++q) {
        const int c = c0 + wn * 64 + 16 * q + 4 * g;
        if (c < a.C) store4(o + static_cast<int64_t>(c) * osize, a.out_type, acc[i][q]);
      }
    } else {
#pragma unroll
      for (int q = 0; q < TC; q += 2) {
        const int c = c0 + wn * 64 + 16 * g + 4 * q;
        if (c < a.C) store8(o + static_cast<int64_t>(c) * osize, a.out_type, acc[i][q], acc[i][q + 1]);
      }
    }
  }
}

// The gradient in the weights: rows are dy's columns n, columns x's columns k,
// and the contraction runs over the expert's positions; both operands are
// stored across it. The rows of perm for a step are loaded a step before its
// data.
template <int TYPE, int BM, int BN, int WM, int WN>
__global__ __launch_bounds__(WM* WN * 64) void k_tile_dw(DwArgs a, int64_t pairs, int run) {
  constexpr int S = 2;
  constexpr int NT = WM * WN * 64;
  constexpr int TR = BM / WM / 16, TC = 4;
  constexpr int NR = BM * 8 / NT, NC = BN * 8 / NT;
  constexpr int RPR = BM / 8, CPR = BN / 8;  // 16-byte pieces of a contraction row
  constexpr int STAGE = (BM + BN) * kStepBytes;
  static_assert(BN == WN * 64 && TR % 4 == 0 && BM >= 128 && BN >= 128, "tile shape");
  __shared__ __attribute__((aligned(16))) char smem[S * STAGE];

  const int64_t pair = pair_of_block(run);
  if (pair >= pairs) return;
  const int n = a.T * a.k;
  const int rtiles = (a.N + BM - 1) / BM, ctiles = (a.K + BN - 1) / BN;
  const int e = static_cast<int>(pair / (static_cast<int64_t>(rtiles) * ctiles));
  const int at = static_cast<int>(pair - static_cast<int64_t>(e) * rtiles * ctiles);
  const int band = at / (8 * ctiles), high = min(8, rtiles - 8 * band), rest = at - band * 8 * ctiles;
  const int r0 = (8 * band + rest % high) * BM, c0 = rest / high * BN;
  const int lo = n > 0 ? min(max(a.offsets[e], 0), n) : 0;
  const int count = n > 0 ? max(min(max(a.offsets[e + 1], 0), n) - lo, 0) : 0;

  const int tid = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int g = lane >> 4, j = lane & 15;
  const int steps = (count + 63) / 64, full = count / 64;

  int rcol[NR], ccol[NC];
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int col = r0 + ((tid % RPR) ^ swz_q(i * (NT / RPR) + tid / RPR)) * 8;
    rcol[i] = col < a.N ? col : r0;
  }
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int col = c0 + ((tid % CPR) ^ swz_q(i * (NT / CPR) + tid / CPR)) * 8;
    ccol[i] = col < a.K ? col : c0;
  }
  int rrow[NR], crow[NC];  // source rows of the next step to be issued
  auto look_up = [&](int kb) {
    if (kb >= steps) return;
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const int p = lo + min(kb * 64 + i * (NT / RPR) + tid / RPR, count - 1);
      rrow[i] = max(row_of(a.perm, a.dy_order, a.k, n, p, a.err), 0);
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int p = lo + min(kb * 64 + i * (NT / CPR) + tid / CPR, count - 1);
      crow[i] = max(row_of(a.perm, a.x_order, a.k, n, p, a.err), 0);
    }
  };
  auto issue = [&](int kb) {
    char* sr = smem + (kb % S) * STAGE + wave * 1024;
    char* sc = sr + BM * kStepBytes;
    const uint16_t* dy = static_cast<const uint16_t*>(a.dy);
    const uint16_t* x = static_cast<const uint16_t*>(a.x);
    const u32x4_t zero = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      if (kb < full || kb * 64 + i * (NT / RPR) + tid / RPR < count)
        load_lds16(dy + static_cast<int64_t>(rrow[i]) * a.N + rcol[i], sr + i * NT * 16);
      else
        *reinterpret_cast<u32x4_t*>(sr + i * NT * 16 + lane * 16) = zero;
    }
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      if (kb < full || kb * 64 + i * (NT / CPR) + tid / CPR < count)
        load_lds16(x + static_cast<int64_t>(crow[i]) * a.K + ccol[i], sc + i * NT * 16);
      else
        *reinterpret_cast<u32x4_t*>(sc + i * NT * 16 + lane * 16) = zero;
    }
  };

  f32x4_t acc[TR][TC];
#pragma unroll
  for (int i = 0; i < TR; ++i)
#pragma unroll
    for (int q = 0; q < TC; ++q) acc[i][q] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  const int q0 = 8 * g + (j >> 2), sw = swz_q(q0);
  int ra[TR], ca[TC];
#pragma unroll
  for (int i = 0; i < TR; ++i)
    ra[i] = lds_address(smem) + q0 * BM * 2 + (((wm * TR * 16 + 16 * i) / 8 + ((j & 3) >> 1)) ^ sw) * 16 + (j & 1) * 8;
#pragma unroll
  for (int i = 0; i < TC; ++i)
    ca[i] = lds_address(smem) + BM * kStepBytes + q0 * BN * 2 + (((wn * 64 + 16 * i) / 8 + ((j & 3) >> 1)) ^ sw) * 16 +
            (j & 1) * 8;

  auto half = [&](int st, auto h_) {
    constexpr int H = decltype(h_)::value;
    u32x4_t cf[TC];
    int at4[4];
#pragma unroll
    for (int q = 0; q < TC; ++q) at4[q] = ca[q] + st;
    lds_tr_x4<H * 64 * BN, H * 64 * BN + 8 * BN>(at4, cf);
#pragma unroll
    for (int i = 0; i < TR; i += 4) {
      u32x4_t rf[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) at4[q] = ra[i + q] + st;
      lds_tr_x4<H * 64 * BM, H * 64 * BM + 8 * BM>(at4, rf);
#pragma unroll
      for (int v = 0; v < 4; ++v)
#pragma unroll
        for (int q = 0; q < TC; ++q) acc[i + v][q] = mma16<TYPE>(cf[q], rf[v], acc[i + v][q]);
    }
  };

  look_up(0);
  if (steps > 0) issue(0);
  look_up(1);
  for (int kb = 0; kb < steps; ++kb) {
    barrier_keep<0>();
    if (kb + 1 < steps) issue(kb + 1);
    look_up(kb + 2);
    half((kb % S) * STAGE, std::integral_constant<int, 0>{});
    half((kb % S) * STAGE, std::integral_constant<int, 1>{});
  }

  const int osize = a.out_type == 1 ? 4 : 2;
#pragma unroll
  for (int i = 0; i < TR; ++i) {
    const int r = r0 + wm * TR * 16 + 16 * i + j;
    if (r >= a.N) continue;
    char* o = static_cast<char*>(a.out) + (static_cast<int64_t>(e) * a.N + r) * a.K * osize;
#pragma unroll
    for (int q = 0; q < TC; ++q) {
      const int c = c0 + wn * 64 + 16 * q + 4 * g;
      if (c < a.K) store4(o + static_cast<int64_t>(c) * osize, a.out_type, acc[i][q]);
    }
  }
}

template <int TYPE, int BM, int BN, int WM, int WN, int S, bool CT>
hipError_t launch_tiles(const ProductArgs& a, hipStream_t s) {
  const int64_t n = static_cast<int64_t>(a.T) * a.k;
  const int64_t ctiles = (a.C + BN - 1) / BN;
  // row tiles: every bucket's last one may be partial
  const int64_t pairs = (a.offsets ? n / BM + std::min<int64_t>(a.E, n) : (n + BM - 1) / BM) * ctiles;
  const int run = static_cast<int>(std::min<int64_t>(32, (pairs + 7) / 8));
  const int64_t grid = (pairs + 8 * run - 1) / (8 * run) * (8 * run);
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  QSMOE_LAUNCH((k_tile_product<TYPE, BM, BN, WM, WN, S, CT>), dim3(static_cast<unsigned>(grid)), dim3(WM * WN * 64), 0,
               s, a, run);
  return hipGetLastError();
}

template <int TYPE, bool CT>
hipError_t pick_tiles(const ProductArgs& a, hipStream_t s) {
  const int64_t n = static_cast<int64_t>(a.T) * a.k;
  const int64_t mean = n / a.E;
  if (mean >= 192) return launch_tiles<TYPE, 256, 256, 2, 4, 2, CT>(a, s);
  if (mean >= 48) return launch_tiles<TYPE, 128, 256, 2, 4, 3, CT>(a, s);
  return launch_tiles<TYPE, 64, 128, 2, 2, 3, CT>(a, s);
}

template <int TYPE, int BM, int BN, int WM, int WN>
hipError_t launch_dw(const DwArgs& a, hipStream_t s) {
  const int64_t pairs = static_cast<int64_t>(a.E) * ((a.N + BM - 1) / BM) * ((a.K + BN - 1) / BN);
  const int run = static_cast<int>(std::min<int64_t>(32, (pairs + 7) / 8));
  const int64_t grid = (pairs + 8 * run - 1) / (8 * run) * (8 * run);
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  QSMOE_LAUNCH((k_tile_dw<TYPE, BM, BN, WM, WN>), dim3(static_cast<unsigned>(grid)), dim3(WM * WN * 64), 0, s, a,
               pairs, run);
  return hipGetLastError();
}

template <int TYPE>
hipError_t pick_dw(const DwArgs& a, hipStream_t s) {
  const int64_t pairs = static_cast<int64_t>(a.E) * ((a.N + 255) / 256) * ((a.K + 255) / 256);
  if (pairs >= 256) return launch_dw<TYPE, 256, 256, 2, 4>(a, s);
  return launch_dw<TYPE, 128, 128, 2, 2>(a, s);
}

}  // namespace

hipError_t launch_product(const ProductArgs& a, hipStream_t s) {
  if (a.type == kTypeE4m3)
    return a.out_type == 1 ? pick_tiles<kE4m3Wide, false>(a, s) : pick_tiles<kTypeE4m3, false>(a, s);
  if (a.type == 0) return a.transposed ? pick_tiles<0, true>(a, s) : pick_tiles<0, false>(a, s);
  return a.transposed ? pick_tiles<2, true>(a, s) : pick_tiles<2, false>(a, s);
}

hipError_t launch_product_dw(const DwArgs& a, hipStream_t s) {
  return a.type == 0 ? pick_dw<0>(a, s) : pick_dw<2>(a, s);
}

}  // namespace qsmoe

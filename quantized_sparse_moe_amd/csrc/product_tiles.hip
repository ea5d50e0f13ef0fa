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
// lane order), which spreads the 16 rows of a fragment over the banks (no bank
// conflict is counted on any of these kernels). The weights' fragment t takes
// rows 16 (j / 4) + 4 t + j % 4 for j = 0..15, which leaves each lane 16
// consecutive output columns over the 4 fragments. An operand stored across
// the contraction keeps 64 contraction rows of BM or BN values and is read
// with the transposing LDS read.
//
// What bounds it (one MI355X; a large copy moves 4.9 TB/s, a large library
// product reaches 1.44 PFLOP/s in bf16 and 2.75 to 3.15 in FP8):
//   256 x 256, bf16, 8192^3: 0.79 to 0.83 ms, 1.33 to 1.40 PFLOP/s, the matrix
//     cores 69 % busy; FP8, 8192^3: 0.53 to 0.55 ms, 2.0 PFLOP/s, 49 % busy:
//     with reads that all hit L2 it is 10 % less, without the block scales
//     another 9 %; the rest are the barriers of steps of 1 us whose 64 KB per
//     CU take the L2 most of that time.
//   128 x 256, 24576 FP8 rows over 256 experts of 4096 x 4096: 1.06 ms, 4.3
//     TB/s of weights, rows and results, 87 % of the copy's rate; a tile's
//     beginning and end (8 us of 48) is what is left. bf16, 2048 x 4096: 0.86
//     ms, 5.1 TB/s.
//   64 x 128, 512 tokens: 0.75 to 0.77 ms, 5.6 TB/s of weights.
// E4M3 multiplied as bf16 (fp32 and fp16 outputs, fp32 sums) takes half the
// matrix rate and converts its codes on the way: 4096 rows by 4096 x 4096 134
// us against 72, 512 rows 31 against 19, 24576 rows over 256 experts of 4096 x
// 2048 with fp32 outputs in slot order 0.75 ms (3.5 TB/s), 512 tokens 0.46 ms
// (4.8 TB/s).
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

constexpr int kE4m3Wide = 4;  // E4M3 multiplied as bf16: exact products, fp32 sums

template <int TYPE, int BM, int BN, int WM, int WN, int S, bool CT>
__global__ __launch_bounds__(WM* WN * 64) void k_tile_product(ProductArgs a, int run) {
  constexpr bool FP8 = TYPE == kTypeE4m3 || TYPE == kE4m3Wide;
  constexpr int ESIZE = FP8 ? 1 : 2;
  constexpr int NT = WM * WN * 64;
  constexpr int TR = BM / WM / 16;   // row fragments of a wave
  constexpr int TC = BN / WN / 16;   // column fragments
  constexpr int NR = BM * 8 / NT, NC = BN * 8 / NT;
  constexpr int SCALES = FP8 ? WM * WN * 256 : 0;
  constexpr int STAGE = (BM + BN) * kStepBytes + SCALES;
  constexpr int LOADS = NR + NC + (FP8 ? 1 : 0);
  static_assert(TC == 4 && NR >= 1 && NC >= 1 && NT % 256 == 0, "tile shape");
  static_assert(!FP8 || !CT, "FP8 weights have the contraction contiguous");
  __shared__ __attribute__((aligned(16))) char smem[S * STAGE];

  const int n = a.T * a.k;
  const int ctiles = (a.C + BN - 1) / BN;
  TileAt t;
  if (!find_tile<BM>(a.offsets, a.E, n, ctiles, pair_of_block(run), &t)) return;
  const int tid = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int g = lane >> 4, j = lane & 15;
  const int c0 = t.ctile * BN;
  const int qbytes = a.Q * ESIZE;  // <= 2^21
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

  auto issue_full = [&](int kb) {
    char* st = smem + (kb % S) * STAGE;
    char* sr = st + wave * 1024;
    char* sc = sr + BM * kStepBytes;
    const char* cb = cbase + kb * cstep;
#pragma unroll
    for (int i = 0; i < NR; ++i) load_lds16(rp[i] + kb * kStepBytes, sr + i * NT * 16);
#pragma unroll
    for (int i = 0; i < NC; ++i) load_lds16(cb + co[i], sc + i * NT * 16);
    if constexpr (FP8) load_lds4(sp + kb, st + (BM + BN) * kStepBytes + wave * 256);
  };
  auto issue = [&](int kb) {
    if (kb < full) {
      issue_full(kb);
    } else {  // the last step of a ragged contraction: zeros behind its end
      char* st = smem + (kb % S) * STAGE;
      char* sr = st + wave * 1024;
      char* sc = sr + BM * kStepBytes;
      const char* cb = cbase + kb * cstep;
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
      if constexpr (FP8) load_lds4(sp + kb, st + (BM + BN) * kStepBytes + wave * 256);
    }
  };

  f32x4_t acc[TR][TC];
#pragma unroll
  for (int i = 0; i < TR; ++i)
#pragma unroll
    for (int q = 0; q < TC; ++q) acc[i][q] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};

  // fragment addresses within a stage; row fragment i of this wave is the
  // tile's fragment i * WM + wm, so that a short tile leaves both halves less
  int ra[2], ca[TC];
  constexpr int RSTEP = WM * 16 * kStepBytes;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int piece = 4 * h + g;
    ra[h] = (wm * 16 + j) * kStepBytes + (piece ^ swz_r(j)) * 16;
    const int cn = 16 * (j >> 2) + (j & 3);
    if constexpr (!CT) ca[h] = BM * kStepBytes + (wn * TC * 16 + cn) * kStepBytes + (piece ^ swz_c(cn)) * 16;
  }
  if constexpr (CT) {
#pragma unroll
    for (int q = 0; q < TC; ++q)
      ca[q] = BM * kStepBytes + (8 * g + (j >> 2)) * BN * 2 +
              (((wn * TC * 16 + 16 * q) / 8 + ((j & 3) >> 1)) ^ swz_q(8 * g + (j >> 2))) * 16 + (j & 1) * 8;
  }

  // The stage of step kb, once its loads have landed: the S - 2 steps behind
  // it may be in flight, counted only if each issued its full number of loads.
  auto arrive = [&](int kb) {
    if (S > 2 && kb + S - 2 < full)
      barrier_keep<(S - 2) * LOADS>();
    else
      barrier_keep<0>();
    if (kb + S - 1 < steps) issue(kb + S - 1);
  };
  auto stage_of = [&](int kb) -> const char* { return smem + (kb % S) * STAGE; };
  float sbs = 0.0f;  // the weights' scales of 64 steps, one per lane
  auto weight_scale = [&](int kb) {
    if ((kb & 63) == 0) {
      sbs = csc[min(kb + lane, qb - 1)];
      asm volatile("" ::"v"(sbs));  // wait for it here, not in every step
    }
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(sbs), kb & 63));
  };
  auto frag8 = [&](const char* at0, const char* at1) {
    return __builtin_bit_cast(i32x8_t, __builtin_shufflevector(lds16(at0), lds16(at1), 0, 1, 2, 3, 4, 5, 6, 7));
  };

  // Each step's products over the first 2 * NI row fragments (a tile with few
  // rows skips the others). Fragments are read from LDS one group ahead of
  // their products, across the barrier too: the last group's products run
  // while the next step's first fragments are on their way.
  auto run_steps = [&](auto ni) {
    constexpr int NI = decltype(ni)::value;
    if constexpr (TYPE == kE4m3Wide) {
      for (int kb = 0; kb < steps; ++kb) {
        arrive(kb);
        const char* st = stage_of(kb);
        const float sb = weight_scale(kb);
        const float* ss = reinterpret_cast<const float*>(st + (BM + BN) * kStepBytes) + wm * 16 + j;
        i32x8_t cf[TC];
#pragma unroll
        for (int q = 0; q < TC; ++q) cf[q] = frag8(st + ca[0] + q * 512, st + ca[1] + q * 512);
#pragma unroll
        for (int i = 0; i < 2 * NI; ++i) {
          const i32x8_t rf = frag8(st + ra[0] + i * RSTEP, st + ra[1] + i * RSTEP);
          const float sc = ss[i * WM * 16] * sb;
          u32x4_t rw[4];
#pragma unroll
          for (int v = 0; v < 4; ++v) rw[v] = e4m3_to_bf16x8(rf[2 * v], rf[2 * v + 1]);
#pragma unroll
          for (int q = 0; q < TC; ++q) {
            f32x4_t part = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int v = 0; v < 4; ++v)
              part = mma16<0>(e4m3_to_bf16x8(cf[q][2 * v], cf[q][2 * v + 1]), rw[v], part);
#pragma unroll
            for (int v = 0; v < 4; ++v) acc[i][q][v] = fmaf(part[v], sc, acc[i][q][v]);
          }
        }
      }
    } else if constexpr (FP8) {
      // a block's 128 products are summed by one instruction; its scale is
      // applied one fragment later, just before the next sum takes its place
      constexpr int N = 2 * NI;             // row fragments
      constexpr int NB = N == 4 ? 4 : 3;    // their buffers: fragment 0's is free when the last is multiplied
      i32x8_t cf[TC], rf[NB];
      f32x4_t part[TC];
      float sc[NB], done = 0.0f;
#pragma unroll
      for (int q = 0; q < TC; ++q) part[q] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
      auto cols = [&](const char* st, int q) { cf[q] = frag8(st + ca[0] + q * 512, st + ca[1] + q * 512); };
      auto rows = [&](const char* st, int i) {
        rf[i % NB] = frag8(st + ra[0] + i * RSTEP, st + ra[1] + i * RSTEP);
        sc[i % NB] = reinterpret_cast<const float*>(st + (BM + BN) * kStepBytes)[(i * WM + wm) * 16 + j];
      };
      auto scale = [&](int i, int q) {
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[i][q][v] = fmaf(part[q][v], done, acc[i][q][v]);
        // done here: the compiler would put them off to behind the barrier, with all sums in registers
        asm volatile("" : "+v"(acc[i][q]));
      };
      if (steps > 0) {
        arrive(0);
#pragma unroll
        for (int q = 0; q < TC; ++q) cols(smem, q);
        rows(smem, 0);
      }
      // INNER: the step to be issued is whole, so that nothing branches
      auto step = [&](int kb, auto inner_) {
        constexpr bool INNER = decltype(inner_)::value;
        const bool more = INNER || kb + 1 < steps;
        const float sb = weight_scale(kb);
        const char* st = stage_of(kb);
        const char* next = stage_of(kb + 1);
        rows(st, 1);
        if (N > 2) rows(st, 2);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          const float mine = sc[i % NB] * sb;
          if (i > 0 && i + 2 < N) rows(st, i + 2);
          if (i == N - 2 && more) {
            if constexpr (INNER) {
              barrier_keep<(S - 2) * LOADS>();
              issue_full(kb + S);
            } else {
              arrive(kb + 1);
            }
          }
          if (i == N - 1 && more) rows(next, 0);
#pragma unroll
          for (int q = 0; q < TC; ++q) {
            scale((i + N - 1) % N, q);
            part[q] = mma_fp8(cf[q], rf[i % NB]);
            if (i == N - 1) {
              __builtin_amdgcn_sched_barrier(0);  // the column fragment's registers are free from here on
              if (more) cols(next, q);
            }
          }
          done = mine;
          __builtin_amdgcn_sched_barrier(0);  // or fragments are read far ahead, into registers that spill
        }
      };
      int kb = 0;
      for (; kb + S < full; ++kb) step(kb, std::true_type{});
      for (; kb < steps; ++kb) step(kb, std::false_type{});
#pragma unroll
      for (int q = 0; q < TC; ++q) scale(N - 1, q);
    } else {
      constexpr int N = 2 * NI;           // groups of 2 row fragments in a step: NI for each half of its inputs
      constexpr int NB = N == 4 ? 4 : 3;  // their buffers: group 0's is free when the last is multiplied
      u32x4_t cf[2][TC], rf[NB][2];
      auto cols = [&](const char* st, auto h_) {
        constexpr int H = decltype(h_)::value;
        if constexpr (CT) {
          int at[TC];
#pragma unroll
          for (int q = 0; q < TC; ++q) at[q] = lds_address(st) + ca[q];
          lds_tr_x4<H * 64 * BN, H * 64 * BN + 8 * BN>(at, cf[H]);
        } else {
#pragma unroll
          for (int q = 0; q < TC; ++q) cf[H][q] = lds16(st + ca[H] + q * 512);
        }
      };
      auto rows = [&](const char* st, int it) {
#pragma unroll
        for (int v = 0; v < 2; ++v) rf[it % NB][v] = lds16(st + ra[it / NI] + ((it % NI) * 2 + v) * RSTEP);
      };
      const std::integral_constant<int, 0> first;
      const std::integral_constant<int, 1> second;
      if (steps > 0) {
        arrive(0);
        cols(smem, first);
        rows(smem, 0);
      }
      auto step = [&](int kb, auto inner_) {
        constexpr bool INNER = decltype(inner_)::value;
        const bool more = INNER || kb + 1 < steps;
        const char* st = stage_of(kb);
        const char* next = stage_of(kb + 1);
        rows(st, 1);
        if (N > 2) rows(st, 2);
        if (N == 2) cols(st, second);
#pragma unroll
        for (int it = 0; it < N; ++it) {
          if (N > 2 && it + 1 == NI) cols(st, second);
          if (it > 0 && it + 2 < N) rows(st, it + 2);
          // the stage's last reads are under way: the last two groups are
          // multiplied behind the barrier, while the next stage's first
          // fragments are read
          if (it == N - 2 && more) {
            if constexpr (INNER) {
              barrier_keep<(S - 2) * LOADS>();
              issue_full(kb + S);
            } else {
              arrive(kb + 1);
            }
            if (N > 2 && !CT) cols(next, first);
          }
          if (it == N - 1 && more) {
            if (N == 2 || CT) cols(next, first);
            rows(next, 0);
          }
#pragma unroll
          for (int v = 0; v < 2; ++v)
#pragma unroll
            for (int q = 0; q < TC; ++q) {
              f32x4_t& c = acc[(it % NI) * 2 + v][q];
              c = mma16<TYPE>(cf[it / NI][q], rf[it % NB][v], c);
            }
          __builtin_amdgcn_sched_barrier(0);
        }
      };
      int kb = 0;
      for (; kb + S < full; ++kb) step(kb, std::true_type{});
      for (; kb < steps; ++kb) step(kb, std::false_type{});
    }
  };

#pragma unroll
  for (int s = 0; s < S - 1; ++s)
    if (s < steps) issue(s);
  const int groups = (t.rows + 32 * WM - 1) / (32 * WM);
  if (TR >= 8 && groups >= 4)
    run_steps(std::integral_constant<int, TR / 2>{});
  else if (TR >= 8 && groups == 3)
    run_steps(std::integral_constant<int, TR >= 8 ? 3 : 1>{});
  else if (TR >= 4 && groups >= 2)
    run_steps(std::integral_constant<int, TR >= 4 ? 2 : 1>{});
  else
    run_steps(std::integral_constant<int, 1>{});

  const int osize = a.out_type == 1 ? 4 : 2;
#pragma unroll
  for (int i = 0; i < TR; ++i) {
    const int r = (i * WM + wm) * 16 + j;
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

// Few rows: what bounds the product is reading each weight once, and with few
// tiles the latency of doing so. A workgroup takes 16 RT rows and 16 columns of
// one expert and its 4 waves every fourth step of the contraction each, weights
// and rows straight from memory into registers, a group of steps ahead; their
// sums meet in LDS in a fixed order. One FP8 row by 4096 x 4096: 7.0 us a call,
// which the host's side of it bounds, with one weight again and again or 24 in
// turn (64 x 128 tiles: 17.5 us); six of 256 experts, 101 MB: 23.6 us, 4.3 TB/s
// with other experts in every call, 20.3 us while the last-level cache holds
// the same six.
template <int TYPE, int RT>
__global__ __launch_bounds__(256) void k_split_product(ProductArgs a, int run) {
  constexpr bool FP8 = TYPE == kTypeE4m3 || TYPE == kE4m3Wide;
  constexpr int ESIZE = FP8 ? 1 : 2;
  constexpr int BM = 16 * RT, BN = 16, W = 4;
  constexpr int U = 4 / RT;  // steps of a group
  __shared__ f32x4_t s_sum[W][RT][64];

  const int n = a.T * a.k;
  TileAt t;
  if (!find_tile<BM>(a.offsets, a.E, n, (a.C + BN - 1) / BN, pair_of_block(run), &t)) return;
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, j = lane & 15;
  const int c0 = t.ctile * BN;
  const int qbytes = a.Q * ESIZE;
  const int steps = (qbytes + kStepBytes - 1) / kStepBytes;
  const int qb = (a.Q + 127) / 128;

  // 32 bytes of a column's weights and of a row per lane and step
  const char* wp = static_cast<const char*>(a.c) +
                   (static_cast<int64_t>(t.e) * a.C + min(c0 + j, a.C - 1)) * qbytes + 32 * g;
  const char* rp[RT];
  const float* rs[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int row = max(row_of(a.perm, a.r_order, a.k, n, t.first + min(16 * i + j, t.rows - 1), a.err), 0);
    rp[i] = static_cast<const char*>(a.r) + static_cast<int64_t>(row) * qbytes + 32 * g;
    rs[i] = FP8 ? a.r_scales + static_cast<int64_t>(row) * qb : nullptr;
  }
  const float* cs = FP8 ? a.c_scales + (static_cast<int64_t>(t.e) * ((a.C + 127) / 128) + c0 / 128) * qb : nullptr;

  struct Group {
    u32x4_t w[U][2], r[U][RT][2];
    float s[U][RT];
  };
  auto load = [&](int i, Group& f) {  // the wave's steps 4 i U, ...
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kb = (i * U + u) * W + wave;
      const int rest = qbytes - kb * kStepBytes - 32 * g;  // this lane's bytes from here on
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        f.w[u][h] = u32x4_t{0, 0, 0, 0};
        if (16 * h < rest) f.w[u][h] = *reinterpret_cast<const u32x4_t*>(wp + kb * kStepBytes + 16 * h);
#pragma unroll
        for (int v = 0; v < RT; ++v) {
          f.r[u][v][h] = u32x4_t{0, 0, 0, 0};
          if (16 * h < rest) f.r[u][v][h] = *reinterpret_cast<const u32x4_t*>(rp[v] + kb * kStepBytes + 16 * h);
        }
      }
      if constexpr (FP8) {
        const int b = min(kb, qb - 1);
#pragma unroll
        for (int v = 0; v < RT; ++v) f.s[u][v] = rs[v][b] * cs[b];
      }
    }
  };
  f32x4_t acc[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) acc[i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  auto multiply = [&](int i, const Group& f) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if ((i * U + u) * W + wave >= steps) continue;
#pragma unroll
      for (int v = 0; v < RT; ++v) {
        if constexpr (FP8) {
          f32x4_t part = {0.0f, 0.0f, 0.0f, 0.0f};
          if constexpr (TYPE == kE4m3Wide) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int x = 0; x < 4; x += 2)
                part = mma16<0>(e4m3_to_bf16x8(f.w[u][h][x], f.w[u][h][x + 1]),
                                e4m3_to_bf16x8(f.r[u][v][h][x], f.r[u][v][h][x + 1]), part);
          } else {
            const auto join = [](u32x4_t lo, u32x4_t hi) {
              return __builtin_bit_cast(i32x8_t, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
            };
            part = mma_fp8(join(f.w[u][0], f.w[u][1]), join(f.r[u][v][0], f.r[u][v][1]));
          }
#pragma unroll
          for (int x = 0; x < 4; ++x) acc[v][x] = fmaf(part[x], f.s[u][v], acc[v][x]);
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) acc[v] = mma16<TYPE>(f.w[u][h], f.r[u][v][h], acc[v]);
        }
      }
    }
  };

  const int groups = (steps + W * U - 1) / (W * U);
  Group f[2];
  if (groups > 0) load(0, f[0]);
  for (int i = 0; i < groups; i += 2) {
    if (i + 1 < groups) load(i + 1, f[1]);
    multiply(i, f[0]);
    if (i + 1 < groups) {
      if (i + 2 < groups) load(i + 2, f[0]);
      multiply(i + 1, f[1]);
    }
  }
#pragma unroll
  for (int v = 0; v < RT; ++v) s_sum[wave][v][lane] = acc[v];
  __syncthreads();
  for (int v = wave; v < RT; v += W) {
    f32x4_t sum = s_sum[0][v][lane];
#pragma unroll
    for (int w = 1; w < W; ++w) sum += s_sum[w][v][lane];
    const int r = 16 * v + j, c = c0 + 4 * g;
    if (r >= t.rows || c >= a.C) continue;
    const int row = row_of(a.perm, a.out_order, a.k, n, t.first + r, a.err);
    if (row < 0) continue;
    store4(static_cast<char*>(a.out) + (static_cast<int64_t>(row) * a.C + c) * (a.out_type == 1 ? 4 : 2), a.out_type,
           sum);
  }
}

// The gradient in the weights: rows are dy's columns n, columns x's columns k,
// and the contraction runs over the expert's positions, 32 at a time; both
// operands are stored across it. A bucket is short against the tile (24 steps
// for 768 rows), so what precedes and follows the steps counts: two workgroups
// share a CU (24 KB a stage, at most 256 registers a wave). 24576 bf16 rows
// over 32 experts of 2048 x 4096, fp32 results: 0.57 ms, of which the products
// take 0.39 (1.05 PFLOP/s) and storing 1.07 GB 0.19 (5.5 TB/s); the two barely
// overlap, since a wave alone on its SIMD gains little while the other stores.
// (256 x 256 tiles, one to a CU: 0.73 ms; 128 x 128, three: 0.69.) At 8192^3
// 0.90 ms, 1.23 PFLOP/s.
template <int TYPE, int BM, int BN, bool LOOKUP>
__global__ __launch_bounds__(256, 2) void k_tile_dw(DwArgs a, int64_t pairs, int run) {
  constexpr int S = 3, BK = 32, NT = 256, WM = 2, WN = 2;
  constexpr int TR = BM / WM / 16, TC = BN / WN / 16;
  constexpr int RPR = BM / 8, CPR = BN / 8;              // 16-byte pieces of a contraction row
  constexpr int NR = BK * RPR / NT, NC = BK * CPR / NT;  // pieces of a thread
  constexpr int RB = BK * BM * 2, STAGE = BK * (BM + BN) * 2;
  constexpr int LOADS = NR + NC;
  static_assert(TC == 4 && (TR == 4 || TR == 8) && BM >= 128 && BN >= 128, "tile shape");
  __shared__ __attribute__((aligned(16))) char smem[S * STAGE];

  const int64_t pair = pair_of_block(run);
  if (pair >= pairs) return;
  const int n = a.T * a.k;
  const int rtiles = (a.N + BM - 1) / BM, ctiles = (a.K + BN - 1) / BN;
  const int e = static_cast<int>(pair / (static_cast<int64_t>(rtiles) * ctiles));
  const int at = static_cast<int>(pair - static_cast<int64_t>(e) * rtiles * ctiles);
  // bands of 4 row tiles: a run of 32 pairs is then a square of 1024 x 1024,
  // which reads least (bands of 8: 579 against 572 us, 8192^3 915 against 896)
  const int band = at / (4 * ctiles), high = min(4, rtiles - 4 * band), rest = at - band * 4 * ctiles;
  const int r0 = (4 * band + rest % high) * BM, c0 = rest / high * BN;
  const int lo = n > 0 ? min(max(a.offsets[e], 0), n) : 0;
  const int count = n > 0 ? max(min(max(a.offsets[e + 1], 0), n) - lo, 0) : 0;

  const int tid = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int g = lane >> 4, j = lane & 15;
  const int steps = (count + BK - 1) / BK, full = count / BK;

  // This thread's pieces: contraction rows rq + i * NT / RPR (cq ...), at byte
  // offsets rcol (ccol) of a row. In bucket order a step's rows follow each
  // other, so that the offsets from the step's first row never change; else
  // (LOOKUP) each row is looked up a step ahead.
  const int rq = tid / RPR, cq = tid / CPR;
  const uint32_t rld = a.N * 2, cld = a.K * 2;  // bytes of a row
  uint32_t rcol[NR], ccol[NC];
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int col = r0 + ((tid % RPR) ^ swz_q(rq + i * (NT / RPR))) * 8;
    rcol[i] = (col < a.N ? col : r0) * 2 + (LOOKUP ? 0 : (rq + i * (NT / RPR)) * rld);
  }
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    const int col = c0 + ((tid % CPR) ^ swz_q(cq + i * (NT / CPR))) * 8;
    ccol[i] = (col < a.K ? col : c0) * 2 + (LOOKUP ? 0 : (cq + i * (NT / CPR)) * cld);
  }
  int rraw[NR], craw[NC];  // perm's entries of the step to be issued next
  auto rpos = [&](int kb, int i) { return lo + min(kb * BK + rq + i * (NT / RPR), count - 1); };
  auto cpos = [&](int kb, int i) { return lo + min(kb * BK + cq + i * (NT / CPR), count - 1); };
  auto look_up = [&](int kb) {
    if constexpr (LOOKUP) {
#pragma unroll
      for (int i = 0; i < NR; ++i) rraw[i] = a.perm[rpos(kb, i)];
#pragma unroll
      for (int i = 0; i < NC; ++i) craw[i] = a.perm[cpos(kb, i)];
    }
  };
  uint32_t highest = 0;  // entry, as unsigned: told at the end if it is no assignment
  auto checked = [&](uint32_t raw) {
    highest = max(highest, raw);
    return min(raw, static_cast<uint32_t>(n) - 1);
  };
  const char* dy = static_cast<const char*>(a.dy);
  const char* x = static_cast<const char*>(a.x);
  // Issue step kb into a stage. The next step's rows are looked up before its
  // data, so that waiting for them does not wait for the data.
  auto issue = [&](int kb, int st, auto whole_) {
    char* sr = smem + st + wave * 1024;
    char* sc = sr + RB;
    const char* rp[NR];
    const char* cp[NC];
    if constexpr (LOOKUP) {
      // not before the barrier: the compiler would wait for the look-up there
#pragma unroll
      for (int i = 0; i < NR; ++i) asm volatile("" : "+v"(rraw[i]));
#pragma unroll
      for (int i = 0; i < NC; ++i) asm volatile("" : "+v"(craw[i]));
#pragma unroll
      for (int i = 0; i < NR; ++i)
        rp[i] = dy + rcol[i] + static_cast<uint64_t>(checked(a.dy_order == kBucket ? rpos(kb, i) : rraw[i])) * rld;
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        const uint32_t r = checked(a.x_order == kBucket ? cpos(kb, i) : craw[i]);
        cp[i] = x + ccol[i] + static_cast<uint64_t>(__umulhi(2 * r, a.k_magic) >> a.k_shift) * cld;
      }
      look_up(kb + 1);
    } else {
      const char* dy0 = dy + static_cast<int64_t>(lo + kb * BK) * rld;
      const char* x0 = x + static_cast<int64_t>(lo + kb * BK) * cld;
#pragma unroll
      for (int i = 0; i < NR; ++i) rp[i] = dy0 + rcol[i];
#pragma unroll
      for (int i = 0; i < NC; ++i) cp[i] = x0 + ccol[i];
    }
    if (decltype(whole_)::value || kb < full) {
#pragma unroll
      for (int i = 0; i < NR; ++i) load_lds16(rp[i], sr + i * NT * 16);
#pragma unroll
      for (int i = 0; i < NC; ++i) load_lds16(cp[i], sc + i * NT * 16);
    } else {  // zeros behind the bucket's end
      const u32x4_t zero = {0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        if (kb * BK + rq + i * (NT / RPR) < count)
          load_lds16(rp[i], sr + i * NT * 16);
        else
          *reinterpret_cast<u32x4_t*>(sr + i * NT * 16 + lane * 16) = zero;
      }
#pragma unroll
      for (int i = 0; i < NC; ++i) {
        if (kb * BK + cq + i * (NT / CPR) < count)
          load_lds16(cp[i], sc + i * NT * 16);
        else
          *reinterpret_cast<u32x4_t*>(sc + i * NT * 16 + lane * 16) = zero;
      }
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
    ra[i] = lds_address(smem) + q0 * BM * 2 + (((wm * TR + i) * 2 + ((j & 3) >> 1)) ^ sw) * 16 + (j & 1) * 8;
#pragma unroll
  for (int i = 0; i < TC; ++i)
    ca[i] = lds_address(smem) + RB + q0 * BN * 2 + (((wn * TC + i) * 2 + ((j & 3) >> 1)) ^ sw) * 16 + (j & 1) * 8;

  // Groups of 4 row fragments, each read while the group before it is
  // multiplied, across the barrier too.
  constexpr int G = TR / 4;
  u32x4_t cf[2][TC], rf[2][4];
  auto cols = [&](int st, u32x4_t(&f)[TC]) {
    int at4[4];
#pragma unroll
    for (int q = 0; q < TC; ++q) at4[q] = ca[q] + st;
    lds_tr_x4<0, 8 * BN>(at4, f);
  };
  auto rows = [&](int st, int grp, u32x4_t(&f)[4]) {
    int at4[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) at4[q] = ra[grp * 4 + q] + st;
    lds_tr_x4<0, 8 * BM>(at4, f);
  };
  auto products = [&](int grp, const u32x4_t(&c)[TC], const u32x4_t(&r)[4]) {
#pragma unroll
    for (int v = 0; v < 4; ++v)
#pragma unroll
      for (int q = 0; q < TC; ++q) acc[grp * 4 + v][q] = mma16<TYPE>(c[q], r[v], acc[grp * 4 + v][q]);
  };
  // Step kb reads stage s0 and, across the barrier, the first fragments of the
  // next step from s1; step kb + 3 is issued into s0 behind that barrier. The
  // barrier leaves step kb + 2 in flight where it is whole. INNER: step kb + 3
  // is whole too, so that nothing branches.
  int s0 = 0, s1 = STAGE, s2 = 2 * STAGE;
  auto step = [&](int kb, auto odd_, auto inner_) {
    constexpr int P = decltype(odd_)::value;  // kb % 2
    constexpr bool INNER = decltype(inner_)::value;
    if constexpr (G == 2) {
      rows(s0, 1, rf[1]);
      products(0, cf[P], rf[0]);
    }
    if (INNER || kb + 1 < steps) {
      if (INNER || kb + 2 < full)
        barrier_keep<LOADS>();
      else
        barrier_keep<0>();
      if (INNER || kb + 3 < steps) issue(kb + 3, s0, inner_);
      cols(s1, cf[P ^ 1]);
      rows(s1, 0, rf[G == 2 ? 0 : P ^ 1]);
    }
    if constexpr (G == 2)
      products(1, cf[P], rf[1]);
    else
      products(0, cf[P], rf[P]);
    const int t = s0;
    s0 = s1;
    s1 = s2;
    s2 = t;
  };

  const std::integral_constant<int, 0> even;
  const std::integral_constant<int, 1> odd;
  auto begin = [&](auto whole) {
    look_up(0);
    issue(0, 0, whole);
    if (decltype(whole)::value || steps > 1) issue(1, STAGE, whole);
    if (decltype(whole)::value || 1 < full)
      barrier_keep<LOADS>();
    else
      barrier_keep<0>();
    if (decltype(whole)::value || steps > 2) issue(2, 2 * STAGE, whole);
    cols(0, cf[0]);
    rows(0, 0, rf[0]);
  };
  int kb = 0;
  if (full > 4) {  // a beginning of its own, or the loop waits as if steps before it might be partial
    begin(std::true_type{});
    for (; kb + 4 < full; kb += 2) {
      step(kb, even, std::true_type{});
      step(kb + 1, odd, std::true_type{});
    }
  } else if (steps > 0) {
    begin(std::false_type{});
  }
  for (; kb < steps; kb += 2) {
    step(kb, even, std::false_type{});
    if (kb + 1 < steps) step(kb + 1, odd, std::false_type{});
  }

  if (highest >= static_cast<uint32_t>(n) && count > 0) set_device_error(a.err, 16);
  if (a.out_type == 1) {
#pragma unroll
    for (int i = 0; i < TR; ++i) {
#pragma unroll
      for (int q = 0; q < TC; q += 2) {
        const int c = c0 + (wn * TC + q) * 16;
        store_pair_f32(acc[i][q], acc[i][q + 1], a.K - c, [&](int r) -> float* {
          const int row = r0 + (wm * TR + i) * 16 + r;
          return row < a.N ? static_cast<float*>(a.out) + (static_cast<int64_t>(e) * a.N + row) * a.K + c : nullptr;
        });
      }
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < TR; ++i) {
    const int r = r0 + (wm * TR + i) * 16 + j;
    if (r >= a.N) continue;
    char* o = static_cast<char*>(a.out) + (static_cast<int64_t>(e) * a.N + r) * a.K * 2;
#pragma unroll
    for (int q = 0; q < TC; ++q) {
      const int c = c0 + (wn * TC + q) * 16 + 4 * g;
      if (c < a.K) store4(o + static_cast<int64_t>(c) * 2, a.out_type, acc[i][q]);
    }
  }
}

template <int TYPE, int BM, int BN, int WM, int WN, int S, bool CT>
hipError_t launch_tiles(const ProductArgs& a, hipStream_t s) {
  const int64_t n = static_cast<int64_t>(a.T) * a.k;
  const int64_t ctiles = (a.C + BN - 1) / BN;
  // row tiles: every bucket's last one may be partial
  const int64_t pairs = (a.offsets ? n / BM + std::min<int64_t>(a.E, n) : (n + BM - 1) / BM) * ctiles;
  // runs of an XCD's 32 CUs (24576 bf16 rows over 32 experts: 777 us, with
  // runs of 16 782, of 64 811)
  const int run = static_cast<int>(std::min<int64_t>(32, (pairs + 7) / 8));
  const int64_t grid = (pairs + 8 * run - 1) / (8 * run) * (8 * run);
  if (grid > max_workgroups(WM * WN * 64)) return hipErrorInvalidValue;
  QSMOE_LAUNCH((k_tile_product<TYPE, BM, BN, WM, WN, S, CT>), dim3(static_cast<unsigned>(grid)), dim3(WM * WN * 64), 0,
               s, a, run);
  return hipGetLastError();
}

template <int TYPE, int RT>
hipError_t launch_split(const ProductArgs& a, hipStream_t s) {
  const int64_t n = static_cast<int64_t>(a.T) * a.k;
  const int64_t pairs =
      (a.offsets ? n / (16 * RT) + std::min<int64_t>(a.E, n) : (n + 16 * RT - 1) / (16 * RT)) * ((a.C + 15) / 16);
  const int run = static_cast<int>(std::min<int64_t>(32, (pairs + 7) / 8));
  const int64_t grid = (pairs + 8 * run - 1) / (8 * run) * (8 * run);
  if (grid > max_workgroups(256)) return hipErrorInvalidValue;
  QSMOE_LAUNCH((k_split_product<TYPE, RT>), dim3(static_cast<unsigned>(grid)), dim3(256), 0, s, a, run);
  return hipGetLastError();
}

template <int TYPE, bool CT>
hipError_t pick_tiles(const ProductArgs& a, hipStream_t s) {
  const int64_t n = static_cast<int64_t>(a.T) * a.k;
  const int64_t mean = n / a.E;
  // Row tiles of height h: exact without groups, else every bucket's last one
  // taken as half full (a bucket of fewer rows than h still takes one).
  const int64_t used = std::min<int64_t>(a.E, n);
  auto tiles = [&](int h, int w) {
    const int64_t m = a.offsets ? std::max<int64_t>(used, n / h + (used + 1) / 2) : (n + h - 1) / h;
    return m * ((a.C + w - 1) / w);
  };
  // What a tile size gives was measured on dense FP8 products of 4096 x 4096
  // weights: 256 x 256 0.97 ms per 10^12 products where it fills the chip
  // (128 x 256: 1.2, 128 x 128: 1.3, 64 x 128: 1.6), but one round of tiles
  // takes 59 / 40 / 30 / 19 us however few they are (the last two two to a
  // CU: 47 / 31 us when doubled). So: the largest size whose tiles fill most
  // of the 256 CUs, and for buckets only while rows fill the tile; a grouped
  // product in few rounds of 128 x 256 tiles takes the 128 x 128 ones, which
  // ragged buckets spread better (fp16, 24 buckets of 84 rows: 39 against
  // 55 us), but not with 16-bit inputs and buckets about as high as a tile
  // (bf16, 16 experts of 2048 x 2048, 192 rows each: 60 us against 66, 8 of
  // 4096 x 2048, 160 each: 43 against 47; FP8: 40 against 36).
  if constexpr (!CT) {
    // 16 columns of split contraction. A round of 256 of its workgroups takes
    // 7 / 10 / 15 us for 16 / 32 / 64 rows (FP8, contraction 4096) where one of
    // 64 x 128 tiles takes 18 however few there are: 305 rows by 240 columns 9
    // us against 17, 16 by 8192 12 against 17; where none of the conditions
    // holds it loses, 64 rows by 6144 columns 38 against 19.
    auto parts = [&](int rt) { return tiles(16 * rt, 16); };
    // Buckets of a few rows read each weight once either way, and more waves
    // read them faster (bf16, 8 experts of 2048 x 2048: 4 rows each 14 us
    // against 19, 15 rows 21 against 19; 16 of 512 x 2048: 15 rows 14 against
    // 20).
    if (mean <= 8 && tiles(64, 128) <= 256) return launch_split<TYPE, 1>(a, s);
    if (mean <= 16 && tiles(64, 128) <= 96) return launch_split<TYPE, 1>(a, s);
    if (parts(1) <= 256) return launch_split<TYPE, 1>(a, s);
    if (parts(2) <= 384) return launch_split<TYPE, 2>(a, s);
    if (parts(1) <= 512) return launch_split<TYPE, 1>(a, s);
    if (parts(4) <= 256) return launch_split<TYPE, 4>(a, s);
  }
  if constexpr (TYPE != kE4m3Wide) {
    if (mean >= 192 && tiles(256, 256) >= 192) return launch_tiles<TYPE, 256, 256, 2, 4, 2, CT>(a, s);
  }
  if (mean >= 48) {
    constexpr bool kFp8 = TYPE == kTypeE4m3 || TYPE == kE4m3Wide;
    if (tiles(128, 256) >= (a.offsets && (kFp8 || mean < 120) ? 512 : 192))
      return launch_tiles<TYPE, 128, 256, 2, 4, 3, CT>(a, s);
    if (tiles(128, 128) >= 256) return launch_tiles<TYPE, 128, 128, 2, 2, 2, CT>(a, s);
  }
  return launch_tiles<TYPE, 64, 128, 2, 2, 3, CT>(a, s);
}

template <int TYPE, int BM, int BN>
hipError_t launch_dw(const DwArgs& a, hipStream_t s) {
  const int64_t pairs = static_cast<int64_t>(a.E) * ((a.N + BM - 1) / BM) * ((a.K + BN - 1) / BN);
  // Runs of half of an XCD's 64 workgroups: with 64 all of them work on one
  // expert in lockstep and store together (24576 rows over 32 experts: 690 us
  // with runs of 64, 646 with 32, 670 with 16).
  const int run = static_cast<int>(std::min<int64_t>(32, (pairs + 7) / 8));
  const int64_t grid = (pairs + 8 * run - 1) / (8 * run) * (8 * run);
  if (grid > max_workgroups(256)) return hipErrorInvalidValue;
  if (a.x_order == kBucket && a.dy_order == kBucket)
    QSMOE_LAUNCH((k_tile_dw<TYPE, BM, BN, false>), dim3(static_cast<unsigned>(grid)), dim3(256), 0, s, a, pairs, run);
  else
    QSMOE_LAUNCH((k_tile_dw<TYPE, BM, BN, true>), dim3(static_cast<unsigned>(grid)), dim3(256), 0, s, a, pairs, run);
  return hipGetLastError();
}

// r / d for every r < 2^31 as umulhi(2 r, magic) >> shift: with shift =
// ceil(log2 d) and magic = ceil(2^(31 + shift) / d), the product exceeds
// r * 2^(31 + shift) / d by less than 2^31 <= 2^(31 + shift) / d.
void set_divisor(DwArgs& a) {
  const uint32_t d = a.x_order == kToken ? a.k : 1;
  a.k_shift = 0;
  while ((uint64_t{1} << a.k_shift) < d) ++a.k_shift;
  a.k_magic = static_cast<uint32_t>(((uint64_t{1} << (31 + a.k_shift)) + d - 1) / d);
}

template <int TYPE>
hipError_t pick_dw(DwArgs a, hipStream_t s) {
  set_divisor(a);
  // 256 x 128 tiles from two to a CU on: buckets of 768 rows take 37 us against
  // 41 with 128 x 128 ones at 512 tiles (16 experts of 1024 x 1024), 51 against
  // 53 at 768, 65 against 69 at 1024, 159 against 178 at 2048, but 24 against 21
  // at 256 and 20 against 13 at 8. Short buckets (96 rows) differ by 5 %, and
  // with look-ups the smaller ones are up to 18 % faster between 600 and 900.
  const int64_t pairs = static_cast<int64_t>(a.E) * ((a.N + 255) / 256) * ((a.K + 127) / 128);
  if (pairs >= 512) return launch_dw<TYPE, 256, 128>(a, s);
  return launch_dw<TYPE, 128, 128>(a, s);
}

}  // namespace

hipError_t launch_product(const ProductArgs& a, hipStream_t s) {
  if (a.type == kTypeE4m3)
    return a.out_type != 0 || a.f32_sums ? pick_tiles<kE4m3Wide, false>(a, s) : pick_tiles<kTypeE4m3, false>(a, s);
  if (a.type == 0) return a.transposed ? pick_tiles<0, true>(a, s) : pick_tiles<0, false>(a, s);
  return a.transposed ? pick_tiles<2, true>(a, s) : pick_tiles<2, false>(a, s);
}

hipError_t launch_product_dw(const DwArgs& a, hipStream_t s) {
  return a.type == 0 ? pick_dw<0>(a, s) : pick_dw<2>(a, s);
}

}  // namespace qsmoe

// Products grouped by expert over bf16, fp16 and block-scaled E4M3:
//   out[p][c] = sum_q rows[p][q] * weights[e(p)][c][q]   (or [q][c])
//   dw[e][n][k] = sum over expert e's positions p of dy[p][n] * x[p][k]
// One workgroup per 64 x 64 tile of the output of one expert: 32 contraction
// steps at a time go through LDS as fp32, each thread sums a 4 x 4 square.
#include "common.hpp"
#include "kernels.hpp"

namespace qsmoe {

namespace {

constexpr int kTile = 64, kStep = 32;
enum : int { kBucket = 0, kToken = 1, kSlot = 2 };  // moe_rows

// The row of a matrix in `order` that belongs to bucket position p, or -1
// where perm names a row outside the matrix (which sets the error bit).
__device__ __forceinline__ int row_of(const int32_t* perm, int order, int k, int n, int p, int32_t* err) {
  if (order == kBucket) return p;
  const int a = perm[p];
  if (a < 0 || a >= n) {
    set_device_error(err, 16);
    return -1;
  }
  return order == kToken ? a / k : a;
}

template <int TYPE>
__device__ __forceinline__ float element(const void* m, int64_t i) {
  if constexpr (TYPE == 0) return bf16_to_f32(static_cast<const uint16_t*>(m)[i]);
  if constexpr (TYPE == 2) return f16_to_f32(static_cast<const uint16_t*>(m)[i]);
  if constexpr (TYPE == kTypeE4m3)
    return __builtin_amdgcn_cvt_f32_fp8(static_cast<const uint8_t*>(m)[i], 0);
}

__device__ __forceinline__ void store(void* out, int out_type, int64_t i, float v) {
  if (out_type == 0) static_cast<uint16_t*>(out)[i] = static_cast<uint16_t>(f32_to_bf16_rne(v));
  if (out_type == 1) static_cast<float*>(out)[i] = v;
  if (out_type == 2) static_cast<_Float16*>(out)[i] = static_cast<_Float16>(v);
}

// Tile `tile` of the list of every expert's row tiles: its expert, first
// position and row count. False past the end.
__device__ bool find_tile(const int32_t* offsets, int E, int n, int tile, int* e, int* first, int* rows) {
  for (int i = 0; i < E; ++i) {
    const int lo = offsets ? min(max(offsets[i], 0), n) : 0;
    const int hi = offsets ? min(max(offsets[i + 1], 0), n) : n;
    const int t = (max(hi - lo, 0) + kTile - 1) / kTile;
    if (tile < t) {
      *e = i;
      *first = lo + tile * kTile;
      *rows = min(hi - *first, kTile);
      return true;
    }
    tile -= t;
  }
  return false;
}

__device__ __forceinline__ void multiply(const float (*sr)[kTile + 1], const float (*sc)[kTile + 1], float (&acc)[4][4]) {
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  for (int q = 0; q < kStep; ++q) {
    float r[4], c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      r[i] = sr[q][ty + 16 * i];
      c[i] = sc[q][tx + 16 * i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(r[i], c[j], acc[i][j]);
  }
}

template <int TYPE>
__global__ __launch_bounds__(256) void k_product(ProductArgs a) {
  __shared__ float sr[kStep][kTile + 1], sc[kStep][kTile + 1];
  __shared__ int s_row[kTile];
  const int n = a.T * a.k;
  const int ctiles = (a.C + kTile - 1) / kTile;
  int e, first, rows;
  if (!find_tile(a.offsets, a.E, n, blockIdx.x / ctiles, &e, &first, &rows)) return;
  const int c0 = blockIdx.x % ctiles * kTile;
  if (threadIdx.x < kTile)
    s_row[threadIdx.x] = threadIdx.x < rows ? max(row_of(a.perm, a.r_order, a.k, n, first + threadIdx.x, a.err), 0) : -1;
  const int qb = (a.Q + 127) / 128;
  float acc[4][4] = {};
  for (int q0 = 0; q0 < a.Q; q0 += kStep) {
    __syncthreads();
    for (int i = threadIdx.x; i < kTile * kStep; i += 256) {
      const int t = i / kStep, q = i % kStep;
      float r = 0.0f, c = 0.0f;
      if (q0 + q < a.Q) {
        const int row = s_row[t];
        if (row >= 0) {
          r = element<TYPE>(a.r, static_cast<int64_t>(row) * a.Q + q0 + q);
          if (TYPE == kTypeE4m3) r *= a.r_scales[static_cast<int64_t>(row) * qb + (q0 + q) / 128];
        }
        if (c0 + t < a.C) {
          const int64_t w = static_cast<int64_t>(e) * a.C * a.Q;
          c = element<TYPE>(a.c, w + (a.transposed ? static_cast<int64_t>(q0 + q) * a.C + c0 + t
                                                   : static_cast<int64_t>(c0 + t) * a.Q + q0 + q));
          if (TYPE == kTypeE4m3)
            c *= a.c_scales[(static_cast<int64_t>(e) * ((a.C + 127) / 128) + (c0 + t) / 128) * qb + (q0 + q) / 128];
        }
      }
      sr[q][t] = r;
      sc[q][t] = c;
    }
    __syncthreads();
    multiply(sr, sc, acc);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int t = threadIdx.x / 16 + 16 * i;
    if (t >= rows) continue;
    const int row = row_of(a.perm, a.out_order, a.k, n, first + t, a.err);
    if (row < 0) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = c0 + threadIdx.x % 16 + 16 * j;
      if (c < a.C) store(a.out, a.out_type, static_cast<int64_t>(row) * a.C + c, acc[i][j]);
    }
  }
}

template <int TYPE>
__global__ __launch_bounds__(256) void k_product_dw(DwArgs a) {
  __shared__ float sr[kStep][kTile + 1], sc[kStep][kTile + 1];
  const int n = a.T * a.k;
  const int ktiles = (a.K + kTile - 1) / kTile, ntiles = (a.N + kTile - 1) / kTile;
  const int e = blockIdx.x / ktiles / ntiles;
  const int n0 = blockIdx.x / ktiles % ntiles * kTile, k0 = blockIdx.x % ktiles * kTile;
  const int lo = n > 0 ? min(max(a.offsets[e], 0), n) : 0, hi = n > 0 ? min(max(a.offsets[e + 1], 0), n) : 0;
  float acc[4][4] = {};
  for (int p0 = lo; p0 < hi; p0 += kStep) {
    __syncthreads();
    for (int i = threadIdx.x; i < kTile * kStep; i += 256) {
      const int t = i % kTile, p = p0 + i / kTile;
      float r = 0.0f, c = 0.0f;
      if (p < hi) {
        const int rd = max(row_of(a.perm, a.dy_order, a.k, n, p, a.err), 0);
        const int rx = max(row_of(a.perm, a.x_order, a.k, n, p, a.err), 0);
        if (n0 + t < a.N) r = element<TYPE>(a.dy, static_cast<int64_t>(rd) * a.N + n0 + t);
        if (k0 + t < a.K) c = element<TYPE>(a.x, static_cast<int64_t>(rx) * a.K + k0 + t);
      }
      sr[i / kTile][t] = r;
      sc[i / kTile][t] = c;
    }
    __syncthreads();
    multiply(sr, sc, acc);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int nn = n0 + threadIdx.x / 16 + 16 * i, kk = k0 + threadIdx.x % 16 + 16 * j;
      if (nn < a.N && kk < a.K) store(a.out, a.out_type, (static_cast<int64_t>(e) * a.N + nn) * a.K + kk, acc[i][j]);
    }
}

}  // namespace

hipError_t launch_product(const ProductArgs& a, hipStream_t s) {
  const int n = a.T * a.k;
  const int64_t tiles = (n / kTile + static_cast<int64_t>(min(a.E, n))) * ((a.C + kTile - 1) / kTile);
  if (tiles > INT32_MAX) return hipErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(tiles));
  switch (a.type) {
    case 0: QSMOE_LAUNCH((k_product<0>), grid, dim3(256), 0, s, a); break;
    case 2: QSMOE_LAUNCH((k_product<2>), grid, dim3(256), 0, s, a); break;
    default: QSMOE_LAUNCH((k_product<kTypeE4m3>), grid, dim3(256), 0, s, a); break;
  }
  return hipGetLastError();
}

hipError_t launch_product_dw(const DwArgs& a, hipStream_t s) {
  const int64_t tiles = static_cast<int64_t>(a.E) * ((a.N + kTile - 1) / kTile) * ((a.K + kTile - 1) / kTile);
  if (tiles > INT32_MAX) return hipErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(tiles));
  if (a.type == 0)
    QSMOE_LAUNCH((k_product_dw<0>), grid, dim3(256), 0, s, a);
  else
    QSMOE_LAUNCH((k_product_dw<2>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace qsmoe

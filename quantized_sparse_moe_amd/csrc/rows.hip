// Rows of tokens brought into bucket order and back, with the router's
// weights, and the gradient of the way back. Assignment a = t * k + j is token
// t's j-th; perm (moe_permute) names the assignment of each bucket position,
// positions (moe_invert_perm) the bucket position of each assignment.
//
//   gather        out[p] = w[a] * x[a / k],            a = perm[p]
//   combine       out[t] = sum_j w[t][j] * y[positions[t k + j]]  (+ shared[t])
//   combine grad  dy[p] = w[a] * dout[a / k],  dw[a] = <dout[a / k], y[p]>,
//                                                       p = positions[a]
//
// All in fp32 with one rounding to the output, sums in a fixed order, no
// atomics on values. Memory bounds them; a copy of 1 GiB runs at 5.1 TB/s read plus
// written. 4096 tokens, top-6, rows of 4096 in bf16: gather 35 us (6.7 TB/s of what
// it must move), combine 42 us in slot order and 47 in bucket order (5.6 and 5.0),
// the gradient 85 to 88 us (5.1 to 5.0).
#include <algorithm>

#include "elements.hpp"
#include "kernels.hpp"

namespace qsmoe {

namespace {

// positions[perm[p]] = p, -1 where perm names no position. Each workgroup owns
// kOwned assignments in LDS and reads all of perm: one launch, no atomics on
// memory. An assignment named twice gets its last position. 24576 entries 4.5 us,
// an empty kernel 2.
constexpr int kOwned = 1024, kAtOnce = 6;

__global__ __launch_bounds__(1024) void k_invert_owned(const int32_t* __restrict__ perm, int n, int size,
                                                       int32_t* __restrict__ positions, int32_t* err) {
  __shared__ int32_t owned[kOwned];
  const uint32_t first = blockIdx.x * kOwned, here = min(kOwned, size - static_cast<int>(first));
  owned[threadIdx.x] = -1;
  __syncthreads();
  for (int p0 = 4 * threadIdx.x; p0 < n; p0 += 4 * kAtOnce * 1024) {
    Raw<kF32, 4> r[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const int p = p0 + 4096 * i;
      r[i] = {};
      if (p < n) r[i] = load_raw<kF32, 4>(reinterpret_cast<const char*>(perm + p), n - p);
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int p = p0 + 4096 * i + j;
        const uint32_t a = r[i].w[j];
        if (a - first < here && p < n) atomicMax(&owned[a - first], p);
        if (blockIdx.x == 0 && a + 1 > static_cast<uint32_t>(size) && p < n) set_device_error(err, 16);
      }
    }
  }
  __syncthreads();
  if (threadIdx.x < here) positions[first + threadIdx.x] = owned[threadIdx.x];
}

// Of longer lists every workgroup would read too much: the same in two
// launches, with atomics on memory (a maximum, whose order does not matter).
__global__ __launch_bounds__(256) void k_invert_fill(int size, int32_t* __restrict__ positions) {
  for (int64_t i = blockIdx.x * int64_t{256} + threadIdx.x; i < size; i += gridDim.x * int64_t{256})
    positions[i] = -1;
}
__global__ __launch_bounds__(256) void k_invert_scatter(const int32_t* __restrict__ perm, int n, int size,
                                                        int32_t* __restrict__ positions, int32_t* err) {
  for (int64_t p = blockIdx.x * int64_t{256} + threadIdx.x; p < n; p += gridDim.x * int64_t{256}) {
    const int a = perm[p];
    if (a >= 0 && a < size)
      atomicMax(&positions[a], static_cast<int32_t>(p));
    else if (a != -1)
      set_device_error(err, 16);
  }
}

// Row p of the result for a lane's V elements. ONCE: see store_raw.
template <int IN, int OUT, int V, bool WEIGHTED, bool ONCE>
__device__ __forceinline__ void gather_one(const GatherArgs& g, int64_t p, int at) {
  const int a = g.perm[p];
  if (a < 0 || a >= g.T * g.k) {
    if (a != -1) set_device_error(g.err, 16);
    return;
  }
  const int64_t row = g.slot_order ? a : a / g.k;
  const auto r = load_raw<IN, V>(static_cast<const char*>(g.x) + (row * g.d + at) * kElemBytes<IN>, g.d - at);
  char* to = static_cast<char*>(g.out) + (p * g.d + at) * kElemBytes<OUT>;
  if constexpr (IN == OUT && !WEIGHTED) {
    store_raw<OUT, V, ONCE>(to, r, g.d - at);
  } else {
    float v[V];
    to_f32<IN, V>(r, v);
    if constexpr (WEIGHTED) {
      const float w = g.w[a];
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] *= w;
    }
    store_raw<OUT, V, ONCE>(to, from_f32<OUT, V>(v), g.d - at);
  }
}

template <int IN, int OUT, bool WEIGHTED>
__global__ __launch_bounds__(256) void k_gather(const GatherArgs g, const RowSplit split) {
  constexpr int V = kLaneElems<IN, OUT>;
  for (int64_t b = blockIdx.x; b < split.blocks; b += gridDim.x) {
    int64_t p;
    int at;
    place_of<V>(split, b, &p, &at);
    if (p < g.n && at < g.d) gather_one<IN, OUT, V, WEIGHTED, false>(g, p, at);
  }
}

// A result that no cache holds, where each row of x is read several times.
// Workgroup b runs on XCD b % 8: each XCD takes slices of 2^shift lanes' columns
// one after the other, all rows of a slice together, so that a slice of x (2 MB of
// 4096 rows) stays in its L2, and writes past the caches. 4096 tokens, top-6, rows
// of 4096: 36 us with slices of 32 lanes, 38 with 16, 39 with 64; 61 to 69 row by row,
// 53 with the writes past the caches alone. Where the slices are no multiple of 8, the
// last ones occupy some of the XCDs only: 2304 columns (9 slices) 33 us, row by row 45;
// 2048 20 and 30, 2560 34 and 48, 2880 36 and 54, 5120 53 and 91. Rows that are read
// once gain the writes only: slot order 74 us, row by row 78, top-1 72 and 78. Slices
// that no L2 holds (16384 tokens) 233, row by row 282.
template <int IN, int OUT, bool WEIGHTED>
__global__ __launch_bounds__(256) void k_gather_slices(const GatherArgs g, const int shift, const int slices,
                                                       const int per_slice) {
  constexpr int V = kLaneElems<IN, OUT>;
  const int b = blockIdx.x >> 3, slice = (blockIdx.x & 7) + 8 * (b / per_slice);
  const int64_t p = static_cast<int64_t>(b % per_slice) * (256 >> shift) + (threadIdx.x >> shift);
  const int at = V * ((slice << shift) + (threadIdx.x & ((1 << shift) - 1)));
  if (slice < slices && p < g.n && at < g.d) gather_one<IN, OUT, V, WEIGHTED, true>(g, p, at);
}

// The row of assignment a, -1 for none.
__device__ __forceinline__ int row_at(const int32_t* positions, int a, int n, int32_t* err) {
  if (!positions) return a;
  const int p = positions[a];
  if (p >= 0 && p < n) return p;
  if (p != -1) set_device_error(err, 16);
  return -1;
}

// V elements of a token per lane; the rows of kAhead slots are loaded together
// (4096 tokens, top-6, bucket order: 47 us with 8, 50 with 4).
constexpr int kAhead = 8;

template <int IN, int OUT>
__global__ __launch_bounds__(256) void k_combine_rows(const CombineArgs g, const RowSplit split) {
  constexpr int V = kLaneElems<IN, OUT>;
  for (int64_t b = blockIdx.x; b < split.blocks; b += gridDim.x) {
    int64_t t;
    int at;
    place_of<V>(split, b, &t, &at);
    if (t >= g.T || at >= g.d) continue;
    const int left = g.d - at;
    float acc[V] = {};
    for (int j0 = 0; j0 < g.k; j0 += kAhead) {
      Raw<IN, V> r[kAhead];
      float w[kAhead];
      bool there[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int a = static_cast<int>(t) * g.k + j0 + i;
        const int p = j0 + i < g.k ? row_at(g.positions, a, g.n, g.err) : -1;
        there[i] = p >= 0;
        w[i] = 1.0f;
        if (there[i]) {
          if (g.w) w[i] = g.w[a];
          r[i] = load_raw<IN, V>(
              static_cast<const char*>(g.y) + (static_cast<int64_t>(p) * g.d + at) * kElemBytes<IN>, left);
        }
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (there[i]) {
          float v[V];
          to_f32<IN, V>(r[i], v);
#pragma unroll
          for (int e = 0; e < V; ++e) acc[e] = fmaf(w[i], v[e], acc[e]);
        }
      }
    }
    if (g.shared) {
      float v[V];
      to_f32<IN, V>(load_raw<IN, V>(static_cast<const char*>(g.shared) + (t * g.d + at) * kElemBytes<IN>, left), v);
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] += v[e];
    }
    store_raw<OUT, V>(static_cast<char*>(g.out) + (t * g.d + at) * kElemBytes<OUT>, from_f32<OUT, V>(acc), left);
  }
}

// dy's elements of one lane of 2^shift that step over a row, and the lane's part
// of the inner product.
template <int IN, int DOUT>
__device__ __forceinline__ float combine_grad_row(const CombineGradArgs& g, int64_t a, int p, int lane, int lanes) {
  constexpr int V = kLaneElems<IN, DOUT>;
  const float w = g.w[a];
  const char* dout = static_cast<const char*>(g.dout) + (a / g.k) * g.d * kElemBytes<DOUT>;
  const char* y = static_cast<const char*>(g.y) + static_cast<int64_t>(p) * g.d * kElemBytes<IN>;
  char* dy = static_cast<char*>(g.dy) + static_cast<int64_t>(p) * g.d * kElemBytes<IN>;
  float dot = 0.0f;
#pragma unroll 2
  for (int at = V * lane; at < g.d; at += V * lanes) {
    float u[V], v[V];
    to_f32<DOUT, V>(load_raw<DOUT, V>(dout + at * kElemBytes<DOUT>, g.d - at), u);
    to_f32<IN, V>(load_raw<IN, V>(y + at * kElemBytes<IN>, g.d - at), v);
#pragma unroll
    for (int e = 0; e < V; ++e) {
      dot = fmaf(u[e], v[e], dot);
      u[e] *= w;
    }
    store_raw<IN, V>(dy + at * kElemBytes<IN>, from_f32<IN, V>(u), g.d - at);
  }
  return dot;
}

// 2^shift lanes of a wave per assignment: 4096 tokens, top-8, rows of 64 3.7 us
// (29 with a workgroup each), top-2 of 1003 10.5 (18).
template <int IN, int DOUT>
__global__ __launch_bounds__(256) void k_combine_grad(const CombineGradArgs g, const int shift,
                                                      const int64_t blocks) {
  const int lane = threadIdx.x & ((1 << shift) - 1);
  for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
    const int64_t a = b * (256 >> shift) + (threadIdx.x >> shift);
    const bool there = a < static_cast<int64_t>(g.T) * g.k;
    const int p = there ? row_at(g.positions, static_cast<int>(a), g.n, g.err) : -1;
    float dot = 0.0f;
    if (p >= 0) dot = combine_grad_row<IN, DOUT>(g, a, p, lane, 1 << shift);
    for (int o = 1; o < 1 << shift; o <<= 1) dot += __shfl_xor(dot, o);
    if (there && lane == 0) g.dw[a] = dot;
  }
}

// A workgroup per assignment, where there are few long rows: 366 of 4096 4.5 us,
// 6.8 with a wave each; from 1500 on a wave each is as fast, and with more of them
// faster.
template <int IN, int DOUT>
__global__ __launch_bounds__(256) void k_combine_grad_few(const CombineGradArgs g) {
  __shared__ float part[4];
  const int a = blockIdx.x, p = row_at(g.positions, a, g.n, g.err);
  float dot = 0.0f;
  if (p >= 0) dot = combine_grad_row<IN, DOUT>(g, a, p, threadIdx.x, 256);
  dot = wave_sum(dot);
  if (lane_id() == 0) part[threadIdx.x / 64] = dot;
  __syncthreads();
  if (threadIdx.x == 0) g.dw[a] = (part[0] + part[1]) + (part[2] + part[3]);
}

}  // namespace

hipError_t launch_invert_perm(const int32_t* perm, int n, int size, int32_t* positions, int32_t* err, hipStream_t s) {
  if (std::max(n, size) <= (1 << 16)) {
    QSMOE_LAUNCH(k_invert_owned, dim3((size + kOwned - 1) / kOwned), dim3(1024), 0, s, perm, n, size, positions, err);
    return hipGetLastError();
  }
  QSMOE_LAUNCH(k_invert_fill, dim3(grid_of((size + int64_t{255}) / 256)), dim3(256), 0, s, size, positions);
  if (n > 0)
    QSMOE_LAUNCH(k_invert_scatter, dim3(grid_of((n + int64_t{255}) / 256)), dim3(256), 0, s, perm, n, size, positions,
                 err);
  return hipGetLastError();
}

hipError_t launch_gather_rows(const GatherArgs& g, hipStream_t s) {
  return with_type(g.dtype, [&](auto in) {
    return with_type(g.out_dtype, [&](auto out) {
      constexpr int IN = decltype(in)::value, OUT = decltype(out)::value, V = kLaneElems<IN, OUT>;
      // Slices for every XCD, a result larger than the eight L2s of 4 MB (smaller ones
      // are the next kernel's to find there), and a grid that holds them. Every order,
      // top_k and width measured above gains by it, so the rule asks for none.
      constexpr int shift = 5;
      const int slices = (g.d + (V << shift) - 1) / (V << shift);
      const int per_slice = (g.n + (256 >> shift) - 1) / (256 >> shift);
      const int64_t out_bytes = static_cast<int64_t>(g.n) * g.d * kElemBytes<OUT>;
      const int64_t groups = static_cast<int64_t>((slices + 7) / 8 * 8) * per_slice;
      if (out_bytes > (int64_t{32} << 20) && slices >= 8 && groups <= max_workgroups(256)) {
        const dim3 grid(static_cast<unsigned>(groups));
        if (g.w)
          QSMOE_LAUNCH((k_gather_slices<IN, OUT, true>), grid, dim3(256), 0, s, g, shift, slices, per_slice);
        else
          QSMOE_LAUNCH((k_gather_slices<IN, OUT, false>), grid, dim3(256), 0, s, g, shift, slices, per_slice);
        return hipGetLastError();
      }
      const RowSplit split = split_rows(g.n, g.d, V);
      if (g.w)
        QSMOE_LAUNCH((k_gather<IN, OUT, true>), dim3(grid_of(split.blocks)), dim3(256), 0, s, g, split);
      else
        QSMOE_LAUNCH((k_gather<IN, OUT, false>), dim3(grid_of(split.blocks)), dim3(256), 0, s, g, split);
      return hipGetLastError();
    });
  });
}

hipError_t launch_combine_rows(const CombineArgs& g, hipStream_t s) {
  return with_type(g.dtype, [&](auto in) {
    return with_type(g.out_dtype, [&](auto out) {
      constexpr int IN = decltype(in)::value, OUT = decltype(out)::value;
      const RowSplit split = split_rows(g.T, g.d, kLaneElems<IN, OUT>);
      QSMOE_LAUNCH((k_combine_rows<IN, OUT>), dim3(grid_of(split.blocks)), dim3(256), 0, s, g, split);
      return hipGetLastError();
    });
  });
}

hipError_t launch_combine_rows_grad(const CombineGradArgs& g, hipStream_t s) {
  const int assignments = g.T * g.k;
  return with_type(g.dtype, [&](auto in) {
    return with_type(g.dout_dtype, [&](auto dout) {
      constexpr int IN = decltype(in)::value, DOUT = decltype(dout)::value, V = kLaneElems<IN, DOUT>;
      if (g.d > 64 * V && assignments <= 1024) {
        QSMOE_LAUNCH((k_combine_grad_few<IN, DOUT>), dim3(assignments), dim3(256), 0, s, g);
      } else {
        int shift = 0;
        while (shift < 6 && (V << shift) < g.d) ++shift;
        const int64_t blocks = (assignments + int64_t{255 >> shift}) / (256 >> shift);
        QSMOE_LAUNCH((k_combine_grad<IN, DOUT>), dim3(grid_of(blocks)), dim3(256), 0, s, g, shift, blocks);
      }
      return hipGetLastError();
    });
  });
}

}  // namespace qsmoe

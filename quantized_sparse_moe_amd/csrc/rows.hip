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
// atomics on values. Memory bounds them.
#include <algorithm>

#include "elements.hpp"
#include "kernels.hpp"

namespace qsmoe {

namespace {

// positions[perm[p]] = p, -1 where perm names no position. Each workgroup owns
// kOwned assignments in LDS and reads all of perm: one launch, no atomics on
// memory. An assignment named twice gets its last position.
constexpr int kOwned = 1024;

__global__ __launch_bounds__(1024) void k_invert_owned(const int32_t* __restrict__ perm, int n, int size,
                                                       int32_t* __restrict__ positions, int32_t* err) {
  __shared__ int32_t owned[kOwned];
  const int first = blockIdx.x * kOwned;
  owned[threadIdx.x] = -1;
  __syncthreads();
  for (int p0 = threadIdx.x; p0 < n; p0 += 8 * 1024) {
    int a[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = p0 + 1024 * i < n ? perm[p0 + 1024 * i] : -1;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int at = a[i] - first;
      if (at >= 0 && at < kOwned && a[i] < size) atomicMax(&owned[at], p0 + 1024 * i);
      if (blockIdx.x == 0 && (a[i] < -1 || a[i] >= size)) set_device_error(err, 16);
    }
  }
  __syncthreads();
  if (first + static_cast<int>(threadIdx.x) < size) positions[first + threadIdx.x] = owned[threadIdx.x];
}

// Of longer lists every workgroup would read too much: the same in two
// launches, with atomics on memory (a maximum, whose order does not matter).
__global__ __launch_bounds__(256) void k_invert_fill(int size, int32_t* __restrict__ positions) {
  for (int64_t i = blockIdx.x * int64_t{256} + threadIdx.x; i < size; i += gridDim.x * int64_t{256}) positions[i] = -1;
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

// One eight of a row per lane.
template <int IN, int OUT, bool WEIGHTED>
__global__ __launch_bounds__(256) void k_gather(const GatherArgs g, const RowSplit split) {
  const int assignments = g.T * g.k;
  for (int64_t b = blockIdx.x; b < split.blocks; b += gridDim.x) {
    int64_t p;
    int at;
    place_of(split, b, &p, &at);
    if (p >= g.n || at >= g.d) continue;
    const int a = g.perm[p];
    if (a < 0 || a >= assignments) {
      if (a != -1) set_device_error(g.err, 16);
      continue;
    }
    const int64_t row = g.slot_order ? a : a / g.k;
    const Raw8<IN> r = load_raw<IN>(static_cast<const char*>(g.x) + (row * g.d + at) * kElemBytes<IN>, g.d - at);
    char* to = static_cast<char*>(g.out) + (p * g.d + at) * kElemBytes<OUT>;
    if constexpr (IN == OUT && !WEIGHTED) {
      store_raw<OUT>(to, r, g.d - at);
    } else {
      float v[8];
      to_f32<IN>(r, v);
      if constexpr (WEIGHTED) {
        const float w = g.w[a];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= w;
      }
      store_raw<OUT>(to, from_f32<OUT>(v), g.d - at);
    }
  }
}

// The row of assignment a, -1 for none.
__device__ __forceinline__ int row_at(const int32_t* positions, int a, int n, int32_t* err) {
  if (!positions) return a;
  const int p = positions[a];
  if (p >= 0 && p < n) return p;
  if (p != -1) set_device_error(err, 16);
  return -1;
}

// One eight of a token per lane; the rows of kAhead slots are loaded together.
constexpr int kAhead = 4;

template <int IN, int OUT>
__global__ __launch_bounds__(256) void k_combine_rows(const CombineArgs g, const RowSplit split) {
  for (int64_t b = blockIdx.x; b < split.blocks; b += gridDim.x) {
    int64_t t;
    int at;
    place_of(split, b, &t, &at);
    if (t >= g.T || at >= g.d) continue;
    const int left = g.d - at;
    float acc[8] = {};
    for (int j0 = 0; j0 < g.k; j0 += kAhead) {
      Raw8<IN> r[kAhead];
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
          r[i] = load_raw<IN>(static_cast<const char*>(g.y) + (static_cast<int64_t>(p) * g.d + at) * kElemBytes<IN>, left);
        }
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (there[i]) {
          float v[8];
          to_f32<IN>(r[i], v);
#pragma unroll
          for (int e = 0; e < 8; ++e) acc[e] = fmaf(w[i], v[e], acc[e]);
        }
      }
    }
    if (g.shared) {
      float v[8];
      to_f32<IN>(load_raw<IN>(static_cast<const char*>(g.shared) + (t * g.d + at) * kElemBytes<IN>, left), v);
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] += v[e];
    }
    store_raw<OUT>(static_cast<char*>(g.out) + (t * g.d + at) * kElemBytes<OUT>, from_f32<OUT>(acc), left);
  }
}

// One workgroup per assignment.
template <int IN, int DOUT>
__global__ __launch_bounds__(256) void k_combine_grad(const CombineGradArgs g) {
  __shared__ float part[4];
  const int assignments = g.T * g.k;
  for (int64_t a = blockIdx.x; a < assignments; a += gridDim.x) {
    const int p = row_at(g.positions, static_cast<int>(a), g.n, threadIdx.x == 0 ? g.err : nullptr);
    float dot = 0.0f;
    if (p >= 0) {
      const float w = g.w[a];
      const char* dout = static_cast<const char*>(g.dout) + (a / g.k) * g.d * kElemBytes<DOUT>;
      const char* y = static_cast<const char*>(g.y) + static_cast<int64_t>(p) * g.d * kElemBytes<IN>;
      char* dy = static_cast<char*>(g.dy) + static_cast<int64_t>(p) * g.d * kElemBytes<IN>;
      for (int at = 8 * threadIdx.x; at < g.d; at += 8 * 256) {
        float u[8], v[8];
        to_f32<DOUT>(load_raw<DOUT>(dout + static_cast<int64_t>(at) * kElemBytes<DOUT>, g.d - at), u);
        to_f32<IN>(load_raw<IN>(y + static_cast<int64_t>(at) * kElemBytes<IN>, g.d - at), v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          dot = fmaf(u[e], v[e], dot);
          u[e] *= w;
        }
        store_raw<IN>(dy + static_cast<int64_t>(at) * kElemBytes<IN>, from_f32<IN>(u), g.d - at);
      }
    }
    dot = wave_sum(dot);
    if (lane_id() == 0) part[threadIdx.x / 64] = dot;
    __syncthreads();
    if (threadIdx.x == 0) g.dw[a] = (part[0] + part[1]) + (part[2] + part[3]);
    __syncthreads();
  }
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
  const RowSplit split = split_rows(g.n, g.d);
  return with_type(g.dtype, [&](auto in) {
    return with_type(g.out_dtype, [&](auto out) {
      constexpr int IN = decltype(in)::value, OUT = decltype(out)::value;
      if (g.w)
        QSMOE_LAUNCH((k_gather<IN, OUT, true>), dim3(grid_of(split.blocks)), dim3(256), 0, s, g, split);
      else
        QSMOE_LAUNCH((k_gather<IN, OUT, false>), dim3(grid_of(split.blocks)), dim3(256), 0, s, g, split);
      return hipGetLastError();
    });
  });
}

hipError_t launch_combine_rows(const CombineArgs& g, hipStream_t s) {
  const RowSplit split = split_rows(g.T, g.d);
  return with_type(g.dtype, [&](auto in) {
    return with_type(g.out_dtype, [&](auto out) {
      QSMOE_LAUNCH((k_combine_rows<decltype(in)::value, decltype(out)::value>), dim3(grid_of(split.blocks)), dim3(256),
                   0, s, g, split);
      return hipGetLastError();
    });
  });
}

hipError_t launch_combine_rows_grad(const CombineGradArgs& g, hipStream_t s) {
  return with_type(g.dtype, [&](auto in) {
    return with_type(g.dout_dtype, [&](auto dout) {
      QSMOE_LAUNCH((k_combine_grad<decltype(in)::value, decltype(dout)::value>),
                   dim3(grid_of(static_cast<int64_t>(g.T) * g.k)), dim3(256), 0, s, g);
      return hipGetLastError();
    });
  });
}

}  // namespace qsmoe

// SwiGLU between an expert's two products, and its gradient. With gate g and up
// u in the two halves of a row and s = 1 / (1 + e^-g):
//   h  = g s u
//   dg = dh u s (1 + g (1 - s)),   du = dh g s
// fp32 inside, one rounding to the output's type. Memory bounds both.
#include "elements.hpp"
#include "kernels.hpp"

namespace qsmoe {

namespace {

// s and 1 - s. 1 - s = e^-g s keeps its relative accuracy for large g, where
// the difference would cancel. Below g = -64 s is e^g to the last bit, while
// the reciprocal of 1 + e^-g would leave the normal range.
__device__ __forceinline__ void sigmoid_both(float g, float* s, float* t) {
  const bool near = g > -64.0f;
  const float e = expf(near ? -g : g), r = __builtin_amdgcn_rcpf(1.0f + e);
  *s = near ? r : e;
  *t = near ? e * r : 1.0f;
}

template <int DT>
__global__ __launch_bounds__(256) void k_swiglu(const char* __restrict__ gu, int64_t rows, int inner,
                                                char* __restrict__ h, const RowSplit split) {
  for (int64_t b = blockIdx.x; b < split.blocks; b += gridDim.x) {
    int64_t row;
    int at;
    place_of(split, b, &row, &at);
    if (row >= rows || at >= inner) continue;
    const char* p = gu + (2 * row * inner + at) * kElemBytes<DT>;
    const Raw8<DT> rg = load_raw<DT>(p, inner - at);
    const Raw8<DT> ru = load_raw<DT>(p + static_cast<int64_t>(inner) * kElemBytes<DT>, inner - at);
    float g[8], u[8];
    to_f32<DT>(rg, g);
    to_f32<DT>(ru, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float s, t;
      sigmoid_both(g[i], &s, &t);
      u[i] *= g[i] * s;
    }
    store_raw<DT>(h + (row * inner + at) * kElemBytes<DT>, from_f32<DT>(u), inner - at);
  }
}

template <int DT, int DH>
__global__ __launch_bounds__(256) void k_swiglu_grad(const char* __restrict__ gu, const char* __restrict__ dh,
                                                     int64_t rows, int inner, char* __restrict__ dgu,
                                                     const RowSplit split) {
  for (int64_t b = blockIdx.x; b < split.blocks; b += gridDim.x) {
    int64_t row;
    int at;
    place_of(split, b, &row, &at);
    if (row >= rows || at >= inner) continue;
    const int64_t first = (2 * row * inner + at) * kElemBytes<DT>, half = static_cast<int64_t>(inner) * kElemBytes<DT>;
    const Raw8<DT> rg = load_raw<DT>(gu + first, inner - at);
    const Raw8<DT> ru = load_raw<DT>(gu + first + half, inner - at);
    const Raw8<DH> rd = load_raw<DH>(dh + (row * inner + at) * kElemBytes<DH>, inner - at);
    float g[8], u[8], d[8];
    to_f32<DT>(rg, g);
    to_f32<DT>(ru, u);
    to_f32<DH>(rd, d);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float s, t;
      sigmoid_both(g[i], &s, &t);
      u[i] = d[i] * u[i] * s * fmaf(g[i], t, 1.0f);
      d[i] = d[i] * (g[i] * s);
    }
    store_raw<DT>(dgu + first, from_f32<DT>(u), inner - at);
    store_raw<DT>(dgu + first + half, from_f32<DT>(d), inner - at);
  }
}

}  // namespace

hipError_t launch_swiglu(const void* gu, int dtype, int64_t rows, int inner, void* h, hipStream_t s) {
  const RowSplit split = split_rows(rows, inner);
  return with_type(dtype, [&](auto dt) {
    QSMOE_LAUNCH(k_swiglu<decltype(dt)::value>, dim3(grid_of(split.blocks)), dim3(256), 0, s,
                 static_cast<const char*>(gu), rows, inner, static_cast<char*>(h), split);
    return hipGetLastError();
  });
}

hipError_t launch_swiglu_grad(const void* gu, int dtype, const void* dh, int dh_dtype, int64_t rows, int inner,
                              void* dgu, hipStream_t s) {
  const RowSplit split = split_rows(rows, inner);
  return with_type(dtype, [&](auto dt) {
    return with_type(dh_dtype, [&](auto dd) {
      QSMOE_LAUNCH((k_swiglu_grad<decltype(dt)::value, decltype(dd)::value>), dim3(grid_of(split.blocks)), dim3(256),
                   0, s, static_cast<const char*>(gu), static_cast<const char*>(dh), rows, inner,
                   static_cast<char*>(dgu), split);
      return hipGetLastError();
    });
  });
}

}  // namespace qsmoe

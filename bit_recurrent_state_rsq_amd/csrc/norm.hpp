// What the norms of rows (norm.hip, block_norm.hip) share: eight columns of a thread at a time, sums over the
// threads of a row in a fixed order, 8-bit codes.
#pragma once
#include <type_traits>

#include "layer_ops.hpp"

namespace rsq {
namespace {

constexpr int kCols = 8;   // consecutive columns of a thread
enum { kOutF32, kOutBf16, kOutInt8, kOutE4m3 };

template <typename T>
__device__ __forceinline__ void load_cols(const T* p, int c, int cols, bool wide, float (&v)[kCols]) {
  if (wide && c + kCols <= cols) {
    load_vec<kCols>(p + c, v);
  } else {
#pragma unroll
    for (int e = 0; e < kCols; ++e) v[e] = c + e < cols ? to_f32(p[c + e]) : 0.f;
  }
}

template <typename T>
__device__ __forceinline__ void store_cols(T* p, int c, int cols, bool wide, const float (&v)[kCols]) {
  if (wide && c + kCols <= cols) {
    store_vec<kCols>(p + c, v);
  } else {
#pragma unroll
    for (int e = 0; e < kCols; ++e)
      if (c + e < cols) from_f32(v[e], p[c + e]);
  }
}

__device__ __forceinline__ uint32_t max_bits(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Sum (SUM) or the larger bit pattern over the R threads of a row, in a fixed
// order: lanes 1, 2, ... apart, then the wavefronts of the row through LDS.
template <int R, bool SUM>
__device__ __forceinline__ uint32_t row_reduce(uint32_t v, uint32_t* lds) {
  auto join = [](uint32_t a, uint32_t b) {
    if constexpr (SUM) return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    else return max_bits(a, b);
  };
#pragma unroll
  for (int m = 1; m < (R < 64 ? R : 64); m <<= 1) v = join(v, (uint32_t)__shfl_xor((int)v, m, 64));
  if constexpr (R > 64) {
    constexpr int NW = R / 64;
    __syncthreads();   // the last reduction's values have been read
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    v = lds[0];
#pragma unroll
    for (int w = 1; w < NW; ++w) v = join(v, lds[w]);
  }
  return v;
}

// code of y for the step `scale`: zero where the step is zero (or a NaN: the
// scale then says so), clamped to the codes' range
template <int OUT>
__device__ __forceinline__ uint32_t encode(float y, float scale) {
  const float v = scale == 0.f ? 0.f : y / scale;
  if constexpr (OUT == kOutE4m3) {
    return f32_to_e4m3(v);
  } else {
    const float r = rintf(fminf(fmaxf(v, -127.f), 127.f));
    return v == v ? (uint32_t)(int)r & 0xFFu : 0u;
  }
}

// A row's output: values, or codes and their scales (one a row where group is 0).
template <int OUT, int R, int NV>
__device__ __forceinline__ void store_row(const float (&h)[NV][kCols], void* out, float* scales, int64_t row, int64_t stride,
                                          int cols, int group, bool wide, int tid, uint32_t* lds) {
  if constexpr (OUT == kOutF32 || OUT == kOutBf16) {
    typedef typename std::conditional<OUT == kOutF32, float, Bf16>::type O;
    O* y = reinterpret_cast<O*>(out) + row * stride;
#pragma unroll
    for (int i = 0; i < NV; ++i) store_cols(y, (i * R + tid) * kCols, cols, wide, h[i]);
  } else {
    constexpr float qmax = OUT == kOutE4m3 ? 448.f : 127.f;
    // absolute values order like their bit patterns, and a NaN's is the largest
    uint32_t m[NV], all = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      m[i] = 0;
#pragma unroll
      for (int e = 0; e < kCols; ++e) m[i] = max_bits(m[i], __float_as_uint(h[i][e]) & 0x7FFFFFFFu);
      all = max_bits(all, m[i]);
    }
    if (group == 0) all = row_reduce<R, false>(all, lds);
    uint8_t* y = reinterpret_cast<uint8_t*>(out) + row * stride;
    const int groups = group ? cols / group : 1;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * R + tid) * kCols;
      uint32_t g = group ? m[i] : all;
      // a group is group / kCols (4, 8 or 16) neighbouring lanes
      if (group)
        for (int s = 1; s < group / kCols; s <<= 1) g = max_bits(g, (uint32_t)__shfl_xor((int)g, s, 64));
      const float scale = __uint_as_float(g) / qmax;
      if (c < cols) {
        if (group ? c % group == 0 : c == 0) scales[row * groups + (group ? c / group : 0)] = scale;
        uint32_t q[kCols];
#pragma unroll
        for (int e = 0; e < kCols; ++e) q[e] = encode<OUT>(h[i][e], scale);
        if (wide && c + kCols <= cols) {
          *reinterpret_cast<uint2*>(y + c) = make_uint2(q[0] | q[1] << 8 | q[2] << 16 | q[3] << 24,
                                                        q[4] | q[5] << 8 | q[6] << 16 | q[7] << 24);
        } else {
#pragma unroll
          for (int e = 0; e < kCols; ++e)
            if (c + e < cols) y[c + e] = (uint8_t)q[e];
        }
      }
    }
  }
}

}  // namespace
}  // namespace rsq

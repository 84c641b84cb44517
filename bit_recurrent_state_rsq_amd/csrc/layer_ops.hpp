// Element access shared by the operators around the decode step (causal
// convolution, selective scan, attention with decays, norms, 4-bit and 8-bit
// products): fp32 and bf16 activations, eight elements of a thread at a time.
#pragma once
#include "rsq_device.hpp"

namespace rsq {

struct Bf16 {
  uint16_t b;
};

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(Bf16 v) { return bf16_to_f32(v.b); }

// two floats to a bf16 pair (a in the low half), nearest-even; a NaN stays one
__device__ __forceinline__ uint32_t bf16_pair(float a, float b) {
  typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
  bf2 v;
  v[0] = (__bf16)a;
  v[1] = (__bf16)b;
  return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ void from_f32(float v, float& out) { out = v; }
__device__ __forceinline__ void from_f32(float v, Bf16& out) {
  out.b = __builtin_bit_cast(uint16_t, (__bf16)v);
}

// N consecutive elements as N * sizeof(T) / 16 wide accesses. The address is
// 16-byte aligned and N * sizeof(T) a multiple of 16.
template <int N>
__device__ __forceinline__ void load_vec(const float* p, float v[N]) {
#pragma unroll
  for (int i = 0; i < N / 4; ++i) {
    const float4 t = reinterpret_cast<const float4*>(p)[i];
    v[4 * i] = t.x, v[4 * i + 1] = t.y, v[4 * i + 2] = t.z, v[4 * i + 3] = t.w;
  }
}
template <int N>
__device__ __forceinline__ void load_vec(const Bf16* p, float v[N]) {
#pragma unroll
  for (int i = 0; i < N / 8; ++i) {
    const uint4 t = reinterpret_cast<const uint4*>(p)[i];
    const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[8 * i + 2 * q] = __uint_as_float(w[q] << 16);
      v[8 * i + 2 * q + 1] = __uint_as_float(w[q] & 0xFFFF0000u);
    }
  }
}
template <int N>
__device__ __forceinline__ void store_vec(float* p, const float v[N]) {
#pragma unroll
  for (int i = 0; i < N / 4; ++i)
    reinterpret_cast<float4*>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}
template <int N>
__device__ __forceinline__ void store_vec(Bf16* p, const float v[N]) {
#pragma unroll
  for (int i = 0; i < N / 8; ++i)
    reinterpret_cast<uint4*>(p)[i] = make_uint4(bf16_pair(v[8 * i], v[8 * i + 1]), bf16_pair(v[8 * i + 2], v[8 * i + 3]),
                                                bf16_pair(v[8 * i + 4], v[8 * i + 5]), bf16_pair(v[8 * i + 6], v[8 * i + 7]));
}

// [begin, end) of sequence s in the packed rows: offsets[s .. s + 1], or equal
// lengths without offsets. Offsets are device data that the host cannot check,
// so they are clamped into [0, tokens]; an end before its begin is an empty
// sequence, and rows past max_len are not visited.
struct Sequences {
  const int32_t* offsets;
  int64_t tokens;     // rows in all
  int64_t max_len;
  int32_t seqs;
};

__device__ __forceinline__ int64_t seq_range(const Sequences& q, int s, int64_t& len) {
  int64_t b, e;
  if (q.offsets) {
    b = q.offsets[s], e = q.offsets[s + 1];
    b = b < 0 ? 0 : b > q.tokens ? q.tokens : b;
    e = e < b ? b : e > q.tokens ? q.tokens : e;
  } else {
    b = (int64_t)s * q.max_len, e = b + q.max_len;
  }
  len = e - b < q.max_len ? e - b : q.max_len;
  return b;
}

}  // namespace rsq

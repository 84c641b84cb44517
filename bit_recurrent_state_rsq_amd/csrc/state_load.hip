// A dense fp32 state [tiles][d_k][d_v] into a quantized one, as the decode step
// stores its first state: every group gets a fresh step, s = absmax / qmax
// rounded to the step's storage type, and the codes RNE(x RN(1/s)); a zero (or
// infinite) step stores code 0. With the Hadamard rotation each group is
// rotated first; a yoked state's reference takes the dense values; bypass
// columns and window pairs are cleared (none are in use afterwards).
//
// Runs once per prompt: 4 bytes an element read, about 1 written, so bound by
// memory. A lane owns one 8 x 8 chunk, the group / 8 lanes of a scale group are
// neighbours: the code chunks are one lane's to store, the dense rows are read in
// runs of 32 bytes a lane. 128 x 64 heads of 128 x 64 to INT8 (340 MB) take 102 us,
// 3.3 TB/s (a large copy moves 4.9).
#include "host_util.hpp"
#include "rsq_kernels.hpp"

namespace rsq {
namespace {

__device__ void load_chunk_rows(const float* S, int dv, float (&x)[8][8]) {
#pragma unroll
  for (int r = 0; r < 8; ++r) loadf8(S + (size_t)r * dv, x[r]);
}

// unnormalised Walsh-Hadamard transform of a group's row: columns 1, 2, 4 apart
// in the lane, then 8, 16, ... across its lanes, as the decode step's
__device__ void rotate_group(float (&v)[8], int gl, int lane) {
#pragma unroll
  for (int h = 1; h < 8; h <<= 1)
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if ((j & h) == 0) {
        const float lo = v[j], hi = v[j + h];
        v[j] = __fadd_rn(lo, hi);
        v[j + h] = __fsub_rn(lo, hi);
      }
  for (int m = 1; m < gl; m <<= 1)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float p = __shfl_xor(v[j], m, 64);
      v[j] = (lane & m) ? __fsub_rn(p, v[j]) : __fadd_rn(v[j], p);
    }
}

template <int BITS>
__device__ void quantize_chunk(const StepArgs& a, const HeadEntry& he, uint8_t* tb, int i0, int j0, float (&x)[8][8],
                               uint32_t& flags) {
  constexpr int qmax = (1 << (BITS - 1)) - 1;
  const int gl = a.group >> 3, lane = threadIdx.x & 63;
  float s[8];
  int q[8][8];
#pragma unroll
  for (int r = 0; r < 8; ++r) {
    if (a.hadamard) rotate_group(x[r], gl, lane);
    uint32_t m = 0;   // absolute values order like their bit patterns
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, __float_as_uint(x[r][j]) & 0x7FFFFFFFu);
    for (int d = 1; d < gl; d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d, 64));
    const float ratio = __uint_as_float(m) / (float)qmax;
    s[r] = a.scale_f16 ? __half2float(__float2half_rn(ratio)) : ratio;
    const bool finite = s[r] <= 3.4e38f;
    if (!(ratio <= 3.4e38f)) flags |= kStatusNonfinite;
    else if (!finite) flags |= kStatusScaleOverflow;
    const float inv = s[r] > 0.f && finite ? 1.0f / s[r] : 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      // RNE(x inv) of the exact product (rsq_device.hpp); past 2^22 it clamps
      const float t = __builtin_fmaf(x[r][j], inv, kMagic) - kMagic;
      const float c = fminf(fmaxf(t, -(float)(qmax + 1)), (float)qmax);
      if (t != c && t == t) flags |= kStatusClipped;
      q[r][j] = t == t ? (int)c : 0;
    }
  }
  Chunk<BITS> ch;
  pack(q, ch);
  store_chunk<BITS>(tb + ((size_t)(j0 >> 3) * (a.dk >> 3) + (i0 >> 3)) * (8 * BITS), ch);
  // one lane of the group stores the eight rows' steps
  if (((j0 >> 3) & (gl - 1)) == 0)
    store_scales8(a.scale_f16 != 0, tb + he.scales + ((size_t)(j0 / a.group) * a.dk + i0) * (a.scale_f16 ? 2 : 4), s);
}

__global__ __launch_bounds__(256) void state_load_kernel(StepArgs a, const float* dense, int bits32, int yoked) {
  const int tile = blockIdx.x;
  const int bb = tile / a.H, h = tile - bb * a.H;
  const HeadEntry he = head_entry(a, h);
  uint8_t* tb = a.tiles + (size_t)bb * a.batch_stride + he.head_offset;
  const float* S = dense + (size_t)tile * a.dk * a.dv;
  const int cw = a.dv >> 3, chunks = cw * (a.dk >> 3);
  uint32_t flags = 0;
  for (int id = threadIdx.x; id < chunks; id += 256) {
    const int i0 = 8 * (id / cw), j0 = 8 * (id % cw);
    const size_t at = (size_t)(j0 >> 3) * (a.dk >> 3) + (i0 >> 3);
    float x[8][8];
    load_chunk_rows(S + (size_t)i0 * a.dv + j0, a.dv, x);
    if (bits32) {
      store_f32_chunk(tb + at * 256, x);
#pragma unroll
      for (int r = 0; r < 8; ++r)
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (!(fabsf(x[r][j]) <= 3.4e38f)) flags |= kStatusNonfinite;
    } else {
      if (yoked) store_f32_chunk(tb + he.ref + at * 256, x);
      switch (he.bits) {
        case 4: quantize_chunk<4>(a, he, tb, i0, j0, x, flags); break;
        case 6: quantize_chunk<6>(a, he, tb, i0, j0, x, flags); break;
        default: quantize_chunk<8>(a, he, tb, i0, j0, x, flags); break;
      }
    }
  }
  // bypass columns or window pairs: from bypass_u to ref, whole 256-byte sections
  uint4* cols = reinterpret_cast<uint4*>(tb + he.bypass_u);
  for (int i = threadIdx.x; i < (int)((he.ref - he.bypass_u) / 16); i += 256) cols[i] = make_uint4(0, 0, 0, 0);
  if (flags) atomicOr(a.status, flags);
  if (tile == 0 && threadIdx.x == 0) {
    *a.hdr_t = 0;
    *a.hdr_n = 0;
  }
}

}  // namespace

rsq_status launch_state_load(const StepArgs& a, int tiles, const float* dense, bool bits32, bool yoked, void* stream) {
  if (const rsq_status s = check_blocks(tiles, 256)) return s;
  hipLaunchKernelGGL(state_load_kernel, dim3((unsigned)tiles), dim3(256), 0, (hipStream_t)stream, a, dense,
                     bits32 ? 1 : 0, yoked ? 1 : 0);
  return launched("state load");
}

}  // namespace rsq

// Products of a few activation rows with a 4-bit weight matrix,
//   y[m, n] = sum_k x[m, k] code[n, k] scale[n, k / group]  (times x's own scales),
// for the projections around a decode step.
//
// Half a byte a weight against 2 M operations: bound by memory at few rows
// (16 int8 rows x 28672 x 8192, 122 MB: 27.9 us, 4.4 TB/s, where a large copy
// moves 4.9; 1 x 2048 x 4096 is 4.8 us of latency: launch, one round of loads, the
// join), from 32 on by making bf16 numbers of the codes, which the vector unit
// does for each 16 x MT rows anew (64 rows of bf16 76 us).
// The packed layout holds 16 rows x 128 columns in 1 KB, 16 bytes a lane of a
// wavefront's load: lane (g, n) has row n, and its word j the eight codes of
// columns 32 j + 8 g .. + 7, which is what it feeds to the j-th product of 32
// columns. Even columns sit in the low four nibbles and odd ones in the high
// four, so that one mask takes a pair (2 i, 2 i + 1) out of nibbles i, i + 4.
//
// fp32 and bf16 rows: a code c becomes the bf16 number 24 + c (its four bits,
// the sign flipped, are the top mantissa bits at exponent 2^4: shift and one
// three-input bit operation a pair), and 24 sum(x) is subtracted through a
// product of x with the constant -24, the accumulator that every weight tile
// of the group starts from. Products are exact in fp32 (fp32 rows as three
// bf16 pieces); the offset's sums are gone from the accumulator within a group,
// from the leading pieces of fp32 rows within 32 columns.
// int8 rows: int8 products of 16 c (a nibble in the high half of its byte),
// exact in int32. E4M3 rows are bf16 numbers.
//
// A workgroup owns NT tiles of 16 weight rows; its wavefronts take every
// kWaves-th block of 128 columns and join their sums in LDS in a fixed order.
#include "host_util.hpp"
#include "layer_ops.hpp"

namespace rsq {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

enum { kXBf16, kXF32, kXInt8, kXE4m3 };

struct W4Args {
  const void* x;
  const uint8_t* codes;    // packed
  const void* scales;      // [groups][rows], padded
  const float* x_scale;
  void* y;
  int64_t x_stride, y_stride;
  int32_t M, N, K;
  int32_t kblocks, npad;
  int32_t x_groups;        // 0: none, 1: one scale a row, else K / group of them
  int32_t scale_f16, out_bf16;
};

struct PackArgs {
  const int8_t* codes;
  const void* scales;
  uint32_t* out_codes;
  uint8_t* out_scales;
  int32_t N, K, group, scale_size, kblocks, npad;
};

__global__ __launch_bounds__(256) void w4_pack_kernel(PackArgs a) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t words = (int64_t)a.npad * a.kblocks * 16;
  if (id < words) {
    const int j = id & 3, lane = (id >> 2) & 63;
    const int64_t tile = id >> 8;
    const int kb = (int)(tile % a.kblocks);
    const int64_t n = tile / a.kblocks * 16 + (lane & 15);
    const int64_t k = (int64_t)kb * 128 + 32 * j + 8 * (lane >> 4);
    uint32_t w = 0;
    if (n < a.N) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (k + e < a.K) w |= ((uint32_t)a.codes[n * a.K + k + e] & 0xFu) << (4 * ((e >> 1) + 4 * (e & 1)));
    }
    a.out_codes[id] = w;
    return;
  }
  const int64_t s = id - words;
  const int64_t groups = (int64_t)a.kblocks * (128 / a.group);
  if (s >= groups * a.npad) return;
  const int64_t gr = s / a.npad, n = s - gr * a.npad;
  const bool in = n < a.N && gr < a.K / a.group;
  if (a.scale_size == 2)
    reinterpret_cast<uint16_t*>(a.out_scales)[s] = in ? reinterpret_cast<const uint16_t*>(a.scales)[n * (a.K / a.group) + gr] : (uint16_t)0;
  else
    reinterpret_cast<float*>(a.out_scales)[s] = in ? reinterpret_cast<const float*>(a.scales)[n * (a.K / a.group) + gr] : 0.f;
}

constexpr int x_size(int xt) { return xt == kXF32 ? 4 : xt == kXBf16 ? 2 : 1; }

// Memory from a scalar address on, with 32-bit offsets; `bytes` from it are in
// range, where loads outside give zeros. The address is uniform over the workgroup.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* base, uint32_t bytes) {
  const uint64_t p = reinterpret_cast<uint64_t>(base);
  const uint32_t low = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)p);
  const uint32_t high = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(p >> 32));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>((uint64_t)high << 32 | low), 0,
                                           __builtin_amdgcn_readfirstlane((int)bytes), 0x00020000);
}
constexpr int64_t kMaxRowBytes = 1 << 24;   // 32 rows of x then end below 2^30

// Eight consecutive columns of a row of x for one product of 32 columns, as loaded.
template <int XT>
struct XRaw {
  static constexpr int kSize = x_size(XT), kWords = 2 * kSize;
  uint32_t w[kWords];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = 0u;
  }
  // at `offset` (the row's part of it checked against the buffer) + `column` bytes
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t x, uint32_t offset, uint32_t column, bool wide) {
    if (wide) {
      if constexpr (kSize == 1) {
        const auto t = __builtin_amdgcn_raw_buffer_load_b64(x, (int)offset, (int)column, 0);
        w[0] = t[0], w[1] = t[1];
      } else {
#pragma unroll
        for (int i = 0; i < kSize / 2; ++i) {
          const auto t = __builtin_amdgcn_raw_buffer_load_b128(x, (int)(offset + 16 * i), (int)column, 0);
          w[4 * i] = t[0], w[4 * i + 1] = t[1], w[4 * i + 2] = t[2], w[4 * i + 3] = t[3];
        }
      }
    } else {
      zero();
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int at = (int)(offset + e * kSize);
        if constexpr (kSize == 1) w[e >> 2] |= (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(x, at, (int)column, 0) << (8 * (e & 3));
        else if constexpr (kSize == 2) w[e >> 1] |= (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(x, at, (int)column, 0) << (16 * (e & 1));
        else w[e] = __builtin_amdgcn_raw_buffer_load_b32(x, at, (int)column, 0);
      }
    }
  }
};

// ... and as the product takes them
template <int XT>
struct XFrag {
  static constexpr int kPieces = XT == kXF32 ? 3 : 1;
  u32x4 p[kPieces];        // bf16 pieces; int8: words 0 and 1 in the codes' nibble order
};

template <int XT>
__device__ __forceinline__ void convert_x(const XRaw<XT>& r, XFrag<XT>& f) {
  const auto& w = r.w;
  if constexpr (XT == kXBf16) {
    f.p[0] = u32x4{w[0], w[1], w[2], w[3]};
  } else if constexpr (XT == kXF32) {
    // three pieces of the leading 8 bits of what is left hold all 24
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo = __uint_as_float(w[2 * i]), hi = __uint_as_float(w[2 * i + 1]);
#pragma unroll
      for (int q = 0; q < 3; ++q) {
        f.p[q][i] = __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
        lo -= __uint_as_float(__float_as_uint(lo) & 0xFFFF0000u);
        hi -= __uint_as_float(__float_as_uint(hi) & 0xFFFF0000u);
      }
    }
  } else if constexpr (XT == kXInt8) {
    // low nibbles of a code word are columns 0, 4, 1, 5, high ones 2, 6, 3, 7
    f.p[0] = u32x4{__builtin_amdgcn_perm(w[1], w[0], 0x05010400u), __builtin_amdgcn_perm(w[1], w[0], 0x07030602u), 0u, 0u};
  } else {
    float v[8];
    e4m3_bytes4(w[0], v);
    e4m3_bytes4(w[1], v + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      f.p[0][i] = __builtin_amdgcn_perm(__float_as_uint(v[2 * i + 1]), __float_as_uint(v[2 * i]), 0x07060302u);
  }
}

// Codes and scales of NT tiles for a block of 128 columns, as loaded.
template <int GPB, int NT>
struct Block {
  u32x4 w[NT];
  uint32_t s[NT][GPB];
  __device__ __forceinline__ void load(const W4Args& a, __amdgpu_buffer_rsrc_t codes, __amdgpu_buffer_rsrc_t scales,
                                       int tile0, int kb, int lane) {
    const int tiles = a.npad >> 4, ssize = a.scale_f16 ? 2 : 4;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int t = min(i, tiles - 1 - tile0);   // a tile past the last is not stored
      w[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(codes, lane * 16, (t * a.kblocks + kb) * 1024, 0));
#pragma unroll
      for (int q = 0; q < GPB; ++q) {
        const int row = (int)(((uint32_t)(kb * GPB + q) * (uint32_t)a.npad + 16 * t) * ssize);
        s[i][q] = a.scale_f16 ? (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(scales, (lane & 15) * 2, row, 0)
                              : (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(scales, (lane & 15) * 4, row, 0);
      }
    }
  }
  __device__ __forceinline__ float scale(const W4Args& a, int i, int q) const {
    return a.scale_f16 ? __half2float(__ushort_as_half((uint16_t)s[i][q])) : __uint_as_float(s[i][q]);
  }
};

// the eight codes of a word as bf16 numbers 24 + c, in column order
__device__ __forceinline__ u32x4 codes_bf16(uint32_t w) {
  constexpr uint32_t m = 0x00780078u, b = 0x41C041C0u;   // 16 + 8 (sign bit flipped)
  return u32x4{((w << 3) & m) ^ b, ((w >> 1) & m) ^ b, ((w >> 5) & m) ^ b, ((w >> 9) & m) ^ b};
}

__device__ __forceinline__ f32x4 mfma(const u32x4& a, const u32x4& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

template <int XT, int GROUP, int NT, int MT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void w4_kernel(W4Args a) {
  extern __shared__ float part[];   // [WAVES][MT * 16][NT * 16]
  constexpr int GPB = 128 / GROUP, SPG = GROUP / 32;   // groups of a block, products of a group
  constexpr bool INT = XT == kXInt8;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n16 = lane & 15, g = lane >> 4;
  const int tile0 = blockIdx.x * NT;
  const int64_t m0 = (int64_t)blockIdx.y * (16 * MT);
  const bool wide = a.x_stride * x_size(XT) % 16 == 0 && reinterpret_cast<uintptr_t>(a.x) % 16 == 0;

  f32x4 y[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int m = 0; m < MT; ++m) y[i][m] = f32x4{0.f, 0.f, 0.f, 0.f};

  constexpr int size = x_size(XT);
  const int xrow = (int)(a.x_stride * size);
  const int rows = min(a.M - (int)m0, 16 * MT);
  const auto rx = buffer(reinterpret_cast<const uint8_t*>(a.x) + m0 * (int64_t)xrow, (uint32_t)(rows * xrow));
  const auto rw = buffer(a.codes + (size_t)tile0 * a.kblocks * 1024, 0xFFFFFFFFu);
  const auto rs = buffer(reinterpret_cast<const uint8_t*>(a.scales) + (size_t)tile0 * 16 * (a.scale_f16 ? 2 : 4), 0xFFFFFFFFu);
  const uint32_t xoff = (uint32_t)(n16 * xrow + 8 * g * size);
  // the next block's codes, and the next 16 rows of x, are on their way while
  // the last ones are worked on
  Block<GPB, NT> next;
  XRaw<XT> xnext[4];
  auto load_x = [&](int kb, int m) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      // (K is a multiple of 32: a product's columns are all inside or all outside)
      if (kb * 128 + 32 * j < a.K) xnext[j].load(rx, xoff + (uint32_t)(16 * m * xrow), (uint32_t)((kb * 128 + 32 * j) * size), wide);
      else xnext[j].zero();
    }
  };
  if (wave < a.kblocks) {
    next.load(a, rw, rs, tile0, wave, lane);
    load_x(wave, 0);
  }
  for (int kb = wave; kb < a.kblocks; kb += WAVES) {
    const Block<GPB, NT> b = next;
    if (kb + WAVES < a.kblocks) next.load(a, rw, rs, tile0, kb + WAVES, lane);
    const auto& w = b.w;
    float s[NT][GPB];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int q = 0; q < GPB; ++q) s[i][q] = b.scale(a, i, q);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      // (fp32 rows are split group by group: their pieces take more registers)
      XFrag<XT> x[4];
      XRaw<XT> xnow[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (XT == kXF32) xnow[j] = xnext[j];
        else convert_x(xnext[j], x[j]);
      }
      if (m + 1 < MT) load_x(kb, m + 1);
      else if (kb + WAVES < a.kblocks) load_x(kb + WAVES, 0);
#pragma unroll
      for (int q = 0; q < GPB; ++q) {
        if constexpr (XT == kXF32) {
#pragma unroll
          for (int j = 0; j < SPG; ++j) convert_x(xnow[q * SPG + j], x[q * SPG + j]);
        }
        // scales of this lane's four rows of x in this group
        f32x4 xs = {1.f, 1.f, 1.f, 1.f};
        if ((XT == kXInt8 || XT == kXE4m3) && a.x_groups > 1) {
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int64_t row = m0 + 16 * m + 4 * g + r;
            const int gr = kb * GPB + q;
            xs[r] = row < a.M && gr < a.x_groups ? a.x_scale[row * a.x_groups + gr] : 0.f;
          }
        }
        if constexpr (INT) {
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            i32x4 acc = {0, 0, 0, 0};
            constexpr uint32_t hi = 0xF0F0F0F0u;
            if constexpr (SPG == 1) {
              const uint32_t c = w[i][q];
              const uint64_t cb = (uint64_t)((c << 4) & hi) | (uint64_t)(c & hi) << 32;
              const uint64_t xb = (uint64_t)x[q].p[0][0] | (uint64_t)x[q].p[0][1] << 32;
              acc = __builtin_amdgcn_mfma_i32_16x16x32_i8((long)xb, (long)cb, acc, 0, 0, 0);
            } else {
#pragma unroll
              for (int j = 0; j < SPG; j += 2) {
                const uint32_t c0 = w[i][q * SPG + j], c1 = w[i][q * SPG + j + 1];
                const u32x4 cb = {(c0 << 4) & hi, c0 & hi, (c1 << 4) & hi, c1 & hi};
                const u32x4 xb = {x[q * SPG + j].p[0][0], x[q * SPG + j].p[0][1], x[q * SPG + j + 1].p[0][0],
                                  x[q * SPG + j + 1].p[0][1]};
                acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, xb), __builtin_bit_cast(i32x4, cb),
                                                            acc, 0, 0, 0);
              }
            }
            const float sc = s[i][q] * 0.0625f;
#pragma unroll
            for (int r = 0; r < 4; ++r) y[i][m][r] = __builtin_fmaf((float)acc[r], sc * xs[r], y[i][m][r]);
          }
        } else if constexpr (XT == kXF32) {
          // The leading pieces' products of 32 columns each have a sum of their
          // own, so that 24 sum(x) is gone again after one rounding at its size: 16
          // normal rows x 512 x 4736 are off by 8e-8 of the norm (in one sum 8e-7, and
          // fp32 weights in a library's product 6e-7).
          constexpr u32x4 minus24 = {0xC1C0C1C0u, 0xC1C0C1C0u, 0xC1C0C1C0u, 0xC1C0C1C0u};
          const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
          f32x4 start[SPG], rest = zero;
#pragma unroll
          for (int j = 0; j < SPG; ++j) {
            start[j] = mfma(x[q * SPG + j].p[0], minus24, zero);
#pragma unroll
            for (int p = XFrag<XT>::kPieces - 1; p > 0; --p) rest = mfma(x[q * SPG + j].p[p], minus24, rest);
          }
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            f32x4 low = rest, acc[SPG];
#pragma unroll
            for (int j = 0; j < SPG; ++j) {
              const u32x4 c = codes_bf16(w[i][q * SPG + j]);
              acc[j] = mfma(x[q * SPG + j].p[0], c, start[j]);
#pragma unroll
              for (int p = XFrag<XT>::kPieces - 1; p > 0; --p) low = mfma(x[q * SPG + j].p[p], c, low);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              float v = acc[0][r];
#pragma unroll
              for (int j = 1; j < SPG; ++j) v += acc[j][r];
              y[i][m][r] = __builtin_fmaf(v + low[r], s[i][q] * xs[r], y[i][m][r]);
            }
          }
        } else {
          constexpr u32x4 minus24 = {0xC1C0C1C0u, 0xC1C0C1C0u, 0xC1C0C1C0u, 0xC1C0C1C0u};
          f32x4 start = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < SPG; ++j)
#pragma unroll
            for (int p = XFrag<XT>::kPieces - 1; p >= 0; --p) start = mfma(x[q * SPG + j].p[p], minus24, start);
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            f32x4 acc = start;
#pragma unroll
            for (int j = 0; j < SPG; ++j) {
              const u32x4 c = codes_bf16(w[i][q * SPG + j]);
#pragma unroll
              for (int p = XFrag<XT>::kPieces - 1; p >= 0; --p) acc = mfma(x[q * SPG + j].p[p], c, acc);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) y[i][m][r] = __builtin_fmaf(acc[r], s[i][q] * xs[r], y[i][m][r]);
          }
        }
        // (groups one after another: mixed, they hold registers that cost more in
        // resident wavefronts than their order gains)
        if constexpr (MT > 1 || (XT == kXF32 && NT > 2)) __builtin_amdgcn_sched_barrier(0);
      }
    }
  }

  // ---- join the wavefronts' sums; a lane has rows 4 g + r of x and weight row n16
  constexpr int COLS = NT * 16;
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int r = 0; r < 4; ++r) part[(wave * MT * 16 + 16 * m + 4 * g + r) * COLS + 16 * i + n16] = y[i][m][r];
  __syncthreads();
  for (int e = threadIdx.x; e < MT * 16 * COLS; e += 64 * WAVES) {
    const int64_t row = m0 + e / COLS;
    const int col = tile0 * 16 + e % COLS;
    if (row >= a.M || col >= a.N) continue;
    float v = part[e];
#pragma unroll
    for (int q = 1; q < WAVES; ++q) v += part[q * MT * 16 * COLS + e];
    if (a.x_groups == 1) v *= a.x_scale[row];
    if (a.out_bf16) from_f32(v, reinterpret_cast<Bf16*>(a.y)[row * a.y_stride + col]);
    else reinterpret_cast<float*>(a.y)[row * a.y_stride + col] = v;
  }
}

typedef void (*W4Fn)(W4Args);
struct W4Pick {
  W4Fn fn;
  int nt, mt, waves;
};

// Workgroups of NT tiles of weight rows and MT of 16 rows of x. More tiles read
// and convert x fewer times (N / (16 NT)) and the weights fewer times (M / (16 MT),
// all but the first from L2); fewer tiles and more wavefronts put more of the
// chip to work where there are few. By the number of 16 x 16 tiles of y, in us at
// bf16 rows (M x N x K), the shape taken first:
//   below 384    one tile:  1 x 2048 x 4096 4.2, two tiles 5.1, four 6.9
//   to 512       two:       64 x 2048 x 4096 6.7, one 10.3, four 8.1
//   to 1280      four:      16 x 8512 x 2048 5.9, two 6.6, one 8.0; 64 x 4096 x 4096 10.8, two 13.3
//   above        four, four wavefronts: 33 x 8512 x 2048 9.5, eight 10.9; 16 x 28672 x 8192 31.6, 33.9
// There 32 rows of x, 64 and more go two times 16 a workgroup: 32 x 28672 x 8192
// 44, once 16 56; 64 rows 76, 88 (four times 16: 100). Not fp32 rows, whose pieces
// then leave one wavefront a SIMD (64 rows 209, once 16 153), nor bf16 and E4M3
// in groups of 32, which keep a start for every group (256 x 4096 x 4096 39, once
// 16 31).
template <int XT, int GROUP>
W4Pick pick_shape(int M, int tiles) {
  const int64_t mtiles = ceil_div(M, 16), work = tiles * mtiles;
  constexpr int kMost = XT == kXF32 ? 8 : 16;   // (fp32 rows need more registers than sixteen wavefronts leave)
  if (work < 384) return {w4_kernel<XT, GROUP, 1, 1, kMost>, 1, 1, kMost};
  if (work <= 512) return {w4_kernel<XT, GROUP, 2, 1, 8>, 2, 1, 8};
  if (work < 1280) return {w4_kernel<XT, GROUP, 4, 1, 8>, 4, 1, 8};
  constexpr int kRows = XT == kXF32 || (XT != kXInt8 && GROUP == 32) ? 1 : 2;
  if (mtiles == 2 || mtiles >= 4) return {w4_kernel<XT, GROUP, 4, kRows, 4>, 4, kRows, 4};
  return {w4_kernel<XT, GROUP, 4, 1, 4>, 4, 1, 4};
}

template <int XT>
W4Pick pick_group(int group, int M, int tiles) {
  switch (group) {
    case 32: return pick_shape<XT, 32>(M, tiles);
    case 64: return pick_shape<XT, 64>(M, tiles);
    default: return pick_shape<XT, 128>(M, tiles);
  }
}

struct W4Layout {
  int kblocks, npad;
  size_t codes, total;
};

rsq_status w4_layout(int32_t n, int32_t k, int32_t group, int32_t scale_dtype, W4Layout& l) {
  if (n < 1 || k < 1) return fail(RSQ_E_INVALID, "n %d k %d", n, k);
  if (group != 32 && group != 64 && group != 128) return fail(RSQ_E_INVALID, "group %d not in {32, 64, 128}", group);
  if (k % group) return fail(RSQ_E_INVALID, "group %d does not divide k %d", group, k);
  if (scale_dtype != RSQ_F32 && scale_dtype != RSQ_F16) return fail(RSQ_E_INVALID, "scale_dtype %d", scale_dtype);
  // (a workgroup reaches its tiles' codes, and all groups' scales, by 31-bit offsets)
  if (n > (1 << 26) || k > (1 << 22)) return fail(RSQ_E_UNSUPPORTED, "n %d, k %d: above 2^26 or 2^22", n, k);
  l.kblocks = (k + 127) / 128;
  l.npad = (n + 15) / 16 * 16;
  if ((int64_t)l.npad * l.kblocks * 128 > ((int64_t)1 << 34) - 4096)
    return fail(RSQ_E_UNSUPPORTED, "n %d, k %d: 2^34 weights and more", n, k);
  l.codes = (size_t)l.npad * l.kblocks * 64;
  l.total = l.codes + (size_t)l.npad * l.kblocks * (128 / group) * (scale_dtype == RSQ_F16 ? 2 : 4);
  return RSQ_OK;
}

}  // namespace
}  // namespace rsq

using namespace rsq;

extern "C" rsq_status rsq_w4_bytes(int32_t n, int32_t k, int32_t group, int32_t scale_dtype, size_t* bytes) {
  if (!bytes) return fail(RSQ_E_INVALID, "bytes is NULL");
  W4Layout l;
  if (const rsq_status s = w4_layout(n, k, group, scale_dtype, l)) return s;
  *bytes = l.total;
  return RSQ_OK;
}

extern "C" rsq_status rsq_w4_pack(const int8_t* codes, const void* scales, int32_t n, int32_t k, int32_t group,
                                  int32_t scale_dtype, void* packed, size_t packed_bytes, void* stream) {
  W4Layout l;
  if (const rsq_status s = w4_layout(n, k, group, scale_dtype, l)) return s;
  if (!codes || !scales || !packed) return fail(RSQ_E_INVALID, "codes, scales and packed must be non-NULL");
  const int ssize = scale_dtype == RSQ_F16 ? 2 : 4;
  if (!aligned(packed, 16) || !aligned(scales, ssize)) return fail(RSQ_E_INVALID, "packed or scales is not aligned");
  if (packed_bytes < l.total) return fail(RSQ_E_BUFFER, "packed has %zu bytes, the weights need %zu", packed_bytes, l.total);
  const Span written[] = {{packed, (int64_t)l.total, "packed"}};
  const Span read[] = {{codes, (int64_t)n * k, "codes"}, {scales, (int64_t)n * (k / group) * ssize, "scales"}};
  if (const rsq_status s = check_overlap(written, read)) return s;
  PackArgs a{codes, scales, static_cast<uint32_t*>(packed), static_cast<uint8_t*>(packed) + l.codes,
             n, k, group, ssize, l.kblocks, l.npad};
  const int64_t items = (int64_t)l.npad * l.kblocks * (16 + 128 / group);
  if (const rsq_status s = check_blocks(ceil_div(items, 256), 256)) return s;
  hipLaunchKernelGGL(w4_pack_kernel, dim3((unsigned)ceil_div(items, 256)), dim3(256), 0, (hipStream_t)stream, a);
  return launched("4-bit weight packing");
}

extern "C" rsq_status rsq_w4_linear(const rsq_w4* p, void* stream) {
  if (!p) return fail(RSQ_E_INVALID, "w4 is NULL");
  W4Layout l;
  if (const rsq_status s = w4_layout(p->n, p->k, p->group, p->scale_dtype, l)) return s;
  int size;
  switch (p->x_dtype) {
    case RSQ_F32: size = 4; break;
    case RSQ_BF16: size = 2; break;
    case RSQ_INT8: case RSQ_E4M3: size = 1; break;
    default: return fail(RSQ_E_INVALID, "x_dtype %d", p->x_dtype);
  }
  if (p->out_dtype != RSQ_F32 && p->out_dtype != RSQ_BF16) return fail(RSQ_E_INVALID, "out_dtype %d", p->out_dtype);
  if (p->x_group != 0 && (size != 1 || p->x_group != p->group))
    return fail(RSQ_E_INVALID, "x_group %d: 0, or with 8-bit x the weights' group %d", p->x_group, p->group);
  if (p->m < 0 || p->m > 65535 * 16) return fail(RSQ_E_INVALID, "m %d not in [0, %d]", p->m, 65535 * 16);
  if (p->m == 0) return RSQ_OK;   // (an empty tensor has no address)
  if ((size == 1) != (p->x_scale != nullptr)) return fail(RSQ_E_INVALID, "x_scale is given with 8-bit x, and only there");
  if (!p->x || !p->packed || !p->y) return fail(RSQ_E_INVALID, "x, packed and y must be non-NULL");
  if (p->x_stride > kMaxRowBytes / size)
    return fail(RSQ_E_UNSUPPORTED, "rows of x %lld elements apart, more than 2^24 bytes", (long long)p->x_stride);
  if (p->x_stride < p->k || p->y_stride < p->n) return fail(RSQ_E_INVALID, "a row stride is shorter than its row");
  const int osize = p->out_dtype == RSQ_BF16 ? 2 : 4;
  if (!aligned(p->x, size) || !aligned(p->y, osize) || !aligned(p->x_scale, 4) || !aligned(p->packed, 16))
    return fail(RSQ_E_INVALID, "a pointer is not aligned to its element type (packed: 16 bytes)");
  if (p->packed_bytes < l.total)
    return fail(RSQ_E_BUFFER, "packed has %zu bytes, the weights need %zu", p->packed_bytes, l.total);
  const int64_t xg = p->x_scale ? (p->x_group ? p->k / p->group : 1) : 0;
  const Span written[] = {{p->y, span_bytes(p->m, p->y_stride, p->n, osize), "y"}};
  const Span read[] = {{p->x, span_bytes(p->m, p->x_stride, p->k, size), "x"},
                       {p->packed, (int64_t)l.total, "packed"},
                       {p->x_scale, p->m * xg * 4, "x_scale"}};
  if (const rsq_status s = check_overlap(written, read)) return s;
  W4Args a{};
  a.x = p->x;
  a.codes = static_cast<const uint8_t*>(p->packed);
  a.scales = a.codes + l.codes;
  a.x_scale = p->x_scale;
  a.y = p->y;
  a.x_stride = p->x_stride, a.y_stride = p->y_stride;
  a.M = p->m, a.N = p->n, a.K = p->k;
  a.kblocks = l.kblocks, a.npad = l.npad;
  a.x_groups = (int32_t)xg;
  a.scale_f16 = p->scale_dtype == RSQ_F16, a.out_bf16 = p->out_dtype == RSQ_BF16;
  const int tiles = l.npad / 16;
  W4Pick w;
  switch (p->x_dtype) {
    case RSQ_F32: w = pick_group<kXF32>(p->group, p->m, tiles); break;
    case RSQ_BF16: w = pick_group<kXBf16>(p->group, p->m, tiles); break;
    case RSQ_INT8: w = pick_group<kXInt8>(p->group, p->m, tiles); break;
    default: w = pick_group<kXE4m3>(p->group, p->m, tiles); break;
  }
  const dim3 grid((unsigned)ceil_div(tiles, w.nt), (unsigned)ceil_div(p->m, 16 * w.mt));
  const size_t lds = (size_t)w.waves * w.mt * 16 * w.nt * 16 * sizeof(float);   // at most 32 KB
  hipLaunchKernelGGL(w.fn, grid, dim3(64 * w.waves), lds, (hipStream_t)stream, a);
  return launched("4-bit weight product");
}

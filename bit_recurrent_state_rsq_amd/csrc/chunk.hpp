// Pieces, tiles and lane sums shared by the operators that take a prompt in chunks of
// tokens on the matrix cores: the selective scan and attention with the delta rule.
#pragma once
#include "layer_ops.hpp"

namespace rsq {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ f32x4 mfma(const u32x4& a, const u32x4& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// the high halves of two floats as a bf16 pair (a in the low half)
__device__ __forceinline__ uint32_t high_pair(float a, float b) {
  return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}

__device__ __forceinline__ float low_half(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float high_half(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// An fp32 value as N bf16 pieces. Two pieces are each rounded to nearest-even:
// what they leave out is at most 2^-8 of 2^-8 of the value. Three pieces hold all
// 24 bits: each takes the leading 8 of what is left, so the products of pieces are
// exact and their sum is rounded in fp32 only.
template <int N>
__device__ __forceinline__ void split_pair(float a, float b, uint32_t (&p)[N]) {
  if constexpr (N == 2) {
    p[0] = bf16_pair(a, b);
    p[1] = bf16_pair(a - low_half(p[0]), b - high_half(p[0]));
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      p[i] = high_pair(a, b);
      a -= __uint_as_float(__float_as_uint(a) & 0xFFFF0000u);
      b -= __uint_as_float(__float_as_uint(b) & 0xFFFF0000u);
    }
  }
}

// Three pieces of which the first is cut, and so never overflows, and the second rounded: what
// two of them leave is of either sign and at most 2^-16 of the value, where two cut ones leave up
// to 2^-15, always towards zero. The six leading products of such pieces leave out 3.1 x 2^-24 of
// the whole at most, 0.4 in the mean square and nothing in the mean (of cut ones 7.8, 1.5 and 1.1).
__device__ __forceinline__ void split_even(float a, float b, uint32_t (&p)[3]) {
  p[0] = high_pair(a, b);
  a -= __uint_as_float(__float_as_uint(a) & 0xFFFF0000u), b -= __uint_as_float(__float_as_uint(b) & 0xFFFF0000u);
  p[1] = bf16_pair(a, b);
  p[2] = high_pair(a - low_half(p[1]), b - high_half(p[1]));   // (eight bits are left)
}

// A chunk's rows as a buffer: one scalar base, 32-bit offsets, and rows past the
// sequence's end out of its range, where loads give zeros and stores are dropped.
// Offsets of lanes without a row or column of their own start at kOutside. All of
// a loop's loads are unconditional (a chunk past the end has no rows): behind a
// branch the compiler could not tell how many are on their way, and would wait
// for the next chunk's to use this one's.
constexpr uint32_t kOutside = 0x80000000u;
constexpr int64_t kMaxRowBytes = 1 << 24;   // a chunk then ends below 2^30, and nothing wraps
template <int L>   // tokens of a chunk
struct ChunkRows {
  __amdgpu_buffer_rsrc_t rsrc;
  __device__ __forceinline__ ChunkRows(const void* base, int64_t row_bytes, int t0, int len) {
    // uniform over the workgroup
    const uint64_t p = reinterpret_cast<uint64_t>(base) + (uint64_t)(t0 * row_bytes);
    // (the builtin's int goes through uint32_t: it must not extend its sign)
    const uint32_t low = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)p);
    const uint32_t high = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(p >> 32));
    const uint64_t u = (uint64_t)high << 32 | low;
    int rows = min(len - t0, L);
    rows = __builtin_amdgcn_readfirstlane(rows);   // (min and max at once would be a vector instruction)
    rows = max(rows, 0);
    rsrc = __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>(u), 0,
                                             __builtin_amdgcn_readfirstlane((int)(rows * row_bytes)), 0x00020000);
  }
};

// 8 consecutive input elements as PI pieces of 4 words each
template <typename T, int PI>
struct Vec8 {
  u32x4 raw[PI == 1 ? 1 : 2];
  template <int L>
  __device__ __forceinline__ void load(const ChunkRows<L>& r, uint32_t offset) {
#pragma unroll
    for (int i = 0; i < (PI == 1 ? 1 : 2); ++i)
      raw[i] = __builtin_amdgcn_raw_buffer_load_b128(r.rsrc, (int)(offset + 16 * i), 0, 0);
  }
  template <bool EVEN = false>
  __device__ __forceinline__ void pieces(u32x4 (&out)[PI]) const {
    if constexpr (PI == 1) {
      out[0] = raw[0];
    } else {
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t p[PI];
        const float a = __uint_as_float(raw[w >> 1][2 * (w & 1)]), b = __uint_as_float(raw[w >> 1][2 * (w & 1) + 1]);
        if constexpr (EVEN) split_even(a, b, p);
        else split_pair<PI>(a, b, p);
#pragma unroll
        for (int i = 0; i < PI; ++i) out[i][w] = p[i];
      }
    }
  }
  // element e is an infinity or a NaN
  __device__ __forceinline__ bool bad(int e) const {
    if constexpr (PI == 1) return ((raw[0][e >> 1] >> (16 * (e & 1))) & 0x7F80u) == 0x7F80u;
    else return (raw[e >> 2][e & 3] & 0x7F800000u) == 0x7F800000u;
  }
  __device__ __forceinline__ void clear(int e) {
    if constexpr (PI == 1) raw[0][e >> 1] &= (e & 1) ? 0x0000FFFFu : 0xFFFF0000u;
    else raw[e >> 2][e & 3] = 0u;
  }
  // an exponent of all ones carries into the sign's place when one is added
  __device__ __forceinline__ uint32_t bad_bits() const {
    uint32_t t = 0;
#pragma unroll
    for (const auto& r : raw)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        t |= PI == 1 ? (r[i] & 0x7F807F80u) + 0x00800080u : (r[i] & 0x7F800000u) + 0x00800000u;
    return t;
  }
};

typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// A tile in LDS: rows of 2^n 16-byte pieces, none padded. Piece p of row r sits
// at p ^ f(r) of its row, with f such that eight consecutive rows' pairs (2 p,
// 2 p + 1) are in eight different pairs of groups of four banks (transposed
// reads), and the lanes that a fragment's 16-byte reads take together (0-3,
// 12-15, 20-23, 24-27 and the like) are in 16 different groups. Rows of 128
// bytes share the banks with their neighbour, so f then follows from the other
// bits. f goes by the row modulo 16 only, and pieces are joined by exclusive or: a lane has one address for each kind of access, and
// reaches other rows by adding multiples of 16 of them and other pieces by an
// exclusive or with a constant.
template <int ROW>   // elements of a row
struct Tile {
  static constexpr int kBytes = 2 * ROW;
  static __device__ __forceinline__ uint32_t at(int row, int piece) {
    const int r = row ^ ((row >> 1) & 4);
    const int f = ROW >= 128 ? ((r << 1) & 14) | ((row >> 3) & 1) : (r & 6) | ((row >> 3) & 1);
    return (uint32_t)(row * kBytes + ((piece ^ f) << 4));
  }
  // a fragment's piece of row lane % 16: pieces 4 i + lane / 16 (exclusive or 64 i)
  static __device__ __forceinline__ uint32_t fragment(int lane) { return at(lane & 15, lane >> 4); }
  // four elements 4 (lane / 16) of 16 columns of a row (exclusive or 32 a further 16 columns)
  static __device__ __forceinline__ uint32_t four(int row, int lane) {
    return at(row, lane >> 5) + 8 * ((lane >> 4) & 1);
  }
  // Transposed reads (ds_read_b64_tr_b16: in a group of 16 lanes, lane i names
  // the i-th run of four elements and gets the i-th column): lane group g takes
  // rows 4 g .. 4 g + 3 of 16 columns (exclusive or 32 a further 16 columns).
  static __device__ __forceinline__ uint32_t transposed(int lane) {
    const int i = lane & 15;
    return at(4 * (lane >> 4) + (i >> 2), (i >> 1) & 1) + 8 * (i & 1);
  }
};

__device__ __forceinline__ u32x2 read_tr(const uint8_t* p) {
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p));
}

// Contraction index of a k-step of 32 over tokens: lane group g holds tokens
// 4g .. 4g + 3 and 16 + 4g .. 16 + 4g + 3. A product's lanes hold its rows in
// fours like this, so P leaves one product and enters the next in registers.
template <int ROW>
__device__ __forceinline__ u32x4 read_tr8(const uint8_t* p) {
  const u32x2 lo = read_tr(p), hi = read_tr(p + 16 * Tile<ROW>::kBytes);
  return u32x4{lo[0], lo[1], hi[0], hi[1]};
}

// Keeps what is derived from v inside the loop that this stands in: a register
// each for dozens of addresses costs more than the operation that makes them.
__device__ __forceinline__ void local(uint32_t& v) { asm volatile("" : "+v"(v)); }

// One step of a running sum over lanes: the lane that CTRL names, in the rows of
// 16 lanes that ROWS has, zero elsewhere.
template <int CTRL, int ROWS>
__device__ __forceinline__ double scan_step(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, ROWS, 0xF, false);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, ROWS, 0xF, false);
  return v + __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
// sum over the lanes up to this one
__device__ __forceinline__ double wave_scan(double v) {
  v = scan_step<0x111, 0xF>(v);   // row_shr 1, 2, 4, 8
  v = scan_step<0x112, 0xF>(v);
  v = scan_step<0x114, 0xF>(v);
  v = scan_step<0x118, 0xF>(v);
  v = scan_step<0x142, 0xA>(v);   // lane 15 of a row to the next row (rows 1 and 3)
  return scan_step<0x143, 0xC>(v);   // lane 31 to rows 2 and 3
}
__device__ __forceinline__ double lane63(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)b, 63);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(b >> 32), 63);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// A matrix product's result may be read by other instructions only some cycles
// after its issue. The compiler counts them out, but was seen not to across a
// branch, with the result in accumulation registers: the build keeps results out
// of those, and the places where a branch follows wait here besides.
__device__ __forceinline__ void settle() {
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_nop 15");
  __builtin_amdgcn_sched_barrier(0);
}

}  // namespace
}  // namespace rsq

// Products of 8-bit integers with a scale for each token and each channel,
//   y[m, n] = x_scale[m] scale[n] sum_k x[m, k] code[n, k]  (+ bias[n]),
// for the projections of prompts. Sums are exact in int32.
//
// Few rows read the weights: 16 x 12352 x 2048 5.2 to 5.7 us (25 MB, 4.5 to 4.9 TB/s), 32 x 28672 x
// 8192 35 us (6.7 TB/s, some of it from the last-level cache). Many rows are bound by the matrix
// cores and by LDS: 4096 x 28672 x 8192 takes 874 us, 2200 TOP/s, 8192^3 468 us, 2350 TOP/s, where a
// library's int8 product takes 556. A step of 64 columns of a 256 x 256 block is 1024 cycles of
// products on each SIMD, and 96 KB read from LDS and 32 KB written to it, which at 128
// bytes a cycle are as many; four stages of 32 KB leave the loads three steps to arrive.
// A block of 128 x 256 has 512 cycles of products and 88 KB (704 cycles) of LDS, but two of
// them fit a compute unit and shorter rows lose less at their ends: 4096 x 12352 x 2048 115 to 122 us,
// 1750 TOP/s, where the library's product takes 119 to 126.
//
// The weights are laid out once, as products of 16 rows and 64 columns take them:
// 1 KB each, 16 bytes a lane of a wavefront, lane (g, r) columns 16 g .. + 15 of row r.
#include <algorithm>

#include "host_util.hpp"
#include "layer_ops.hpp"

namespace rsq {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

struct W8Args {
  const int8_t* x;
  const uint8_t* codes;   // packed
  const float* scale;     // [N], behind the codes
  const float* x_scale;
  const float* bias;
  void* y;
  int64_t x_stride, y_stride;
  int32_t M, N, K;
  int32_t kblocks, tiles;   // blocks of 64 columns, tiles of 16 rows
  int32_t out_bf16, wide;   // wide: y takes four values at a time
  int32_t mt, nt;           // blocks of the large kernel's grid
};

struct PackArgs {
  const int8_t* codes;
  const float* scales;
  u32x2* out;
  float* out_scales;
  int32_t N, K, kblocks;
  int64_t pieces;
};

// 16 bytes of a row from column k on, zeros from K on; rows may begin at any byte
__device__ __forceinline__ i32x4 row_piece(const int8_t* row, int64_t k, int64_t K) {
  i32x4 v = {0, 0, 0, 0};
  if (k + 16 <= K) {
    __builtin_memcpy(&v, row + k, 16);
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e)
      if (k + e < K) v[e >> 2] |= (int)(uint32_t)(uint8_t)row[k + e] << (8 * (e & 3));
  }
  return v;
}

__global__ __launch_bounds__(256) void w8_pack_kernel(PackArgs a) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id < a.N) a.out_scales[id] = a.scales[id];
  if (id >= a.pieces) return;
  const int lane = id & 63;
  const int64_t block = id >> 6;
  const int64_t n = block / a.kblocks * 16 + (lane & 15);
  const int64_t k = block % a.kblocks * 64 + 16 * (lane >> 4);
  i32x4 v = {0, 0, 0, 0};
  if (n < a.N) v = row_piece(a.codes + n * a.K, k, a.K);
  reinterpret_cast<i32x4*>(a.out)[id] = v;
}

// Four values of a row of y, columns n .. n + 3.
__device__ __forceinline__ void store_four(const W8Args& a, int64_t m, int n, const i32x4& acc, float xs, const float (&ws)[4],
                                           const float (&b)[4]) {
  if (m >= a.M || n >= a.N) return;
  float v[4];
#pragma unroll
  for (int r = 0; r < 4; ++r) v[r] = __builtin_fmaf((float)acc[r] * xs, ws[r], b[r]);
  if (a.out_bf16) {
    uint16_t* y = reinterpret_cast<uint16_t*>(a.y) + m * a.y_stride + n;
    const u32x2 w = {bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
    if (a.wide && n + 4 <= a.N) {
      *reinterpret_cast<u32x2*>(y) = w;
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (n + r < a.N) y[r] = (uint16_t)(w[r >> 1] >> (16 * (r & 1)));
    }
  } else {
    float* y = reinterpret_cast<float*>(a.y) + m * a.y_stride + n;
    if (a.wide && n + 4 <= a.N) {
      *reinterpret_cast<float4*>(y) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (n + r < a.N) y[r] = v[r];
    }
  }
}

__device__ __forceinline__ void load_four(const W8Args& a, int n, float (&ws)[4], float (&b)[4]) {
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const bool in = n + r < a.N;
    ws[r] = in ? a.scale[n + r] : 0.f;
    b[r] = in && a.bias ? a.bias[n + r] : 0.f;
  }
}

// Few rows: bound by reading the weights. A workgroup owns NT tiles of 16 weight rows
// and MT of 16 rows of x; its wavefronts take every WAVES-th block of 64 columns and
// join their sums, which are whole numbers, in LDS.
template <int NT, int MT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void w8_few_kernel(W8Args a) {
  __shared__ __attribute__((aligned(16))) int part[WAVES][NT * MT][64][4];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n16 = lane & 15, g = lane >> 4;
  const int tile0 = blockIdx.x * NT;
  const int64_t m0 = (int64_t)blockIdx.y * (16 * MT);
  i32x4 acc[NT][MT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[i][m] = i32x4{0, 0, 0, 0};
  const int8_t* row[MT];
  bool in[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    in[m] = m0 + 16 * m + n16 < a.M;
    row[m] = a.x + (in[m] ? m0 + 16 * m + n16 : m0) * a.x_stride;
  }
  const uint8_t* w[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) w[i] = a.codes + ((size_t)min(tile0 + i, a.tiles - 1) * a.kblocks * 64 + lane) * 16;
  i32x4 wn[NT], xn[MT];
  auto load = [&](int kb) {
#pragma unroll
    for (int i = 0; i < NT; ++i) wn[i] = *reinterpret_cast<const i32x4*>(w[i] + (size_t)kb * 1024);
#pragma unroll
    for (int m = 0; m < MT; ++m) xn[m] = row_piece(row[m], (int64_t)kb * 64 + 16 * g, a.K);
  };
  if (wave < a.kblocks) load(wave);
  for (int kb = wave; kb < a.kblocks; kb += WAVES) {
    i32x4 wf[NT], xf[MT];
#pragma unroll
    for (int i = 0; i < NT; ++i) wf[i] = wn[i];
#pragma unroll
    for (int m = 0; m < MT; ++m) xf[m] = xn[m];
    if (kb + WAVES < a.kblocks) load(kb + WAVES);
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[i][m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[i], xf[m], acc[i][m], 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int m = 0; m < MT; ++m) *reinterpret_cast<i32x4*>(part[wave][i * MT + m][lane]) = acc[i][m];
  __syncthreads();
  for (int t = wave; t < NT * MT; t += WAVES) {
    i32x4 sum = *reinterpret_cast<const i32x4*>(part[0][t][lane]);
#pragma unroll
    for (int q = 1; q < WAVES; ++q) sum += *reinterpret_cast<const i32x4*>(part[q][t][lane]);
    const int64_t m = m0 + 16 * (t % MT) + n16;
    const int n = (tile0 + t / MT) * 16 + 4 * g;
    float ws[4], b[4];
    load_four(a, n, ws, b);
    store_four(a, m, n, sum, m < a.M ? a.x_scale[m] : 0.f, ws, b);
  }
}

// 16 bytes a lane from memory to LDS, at `lds` (uniform over the wavefront) + 16 lane;
// offsets outside the buffer give zeros. The compiler does not know of these loads.
// (m0 is the compiler's for single instructions only, none of which are used here.)
__device__ __forceinline__ void load_lds(const i32x4& buffer, uint32_t offset, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(__builtin_amdgcn_readfirstlane((int)lds)), "v"(offset), "s"(buffer)
               : "memory");
}

__device__ __forceinline__ i32x4 buffer_of(const void* base, uint32_t bytes) {
  const uint64_t p = reinterpret_cast<uint64_t>(base);
  i32x4 r;
  r[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)p);
  r[1] = __builtin_amdgcn_readfirstlane((int)(uint32_t)(p >> 32) & 0xFFFF);
  r[2] = __builtin_amdgcn_readfirstlane((int)bytes);
  r[3] = 0x00020000;
  return r;
}

constexpr uint32_t kOutside = 0x80000000u;

// Many rows: BM x BN of y a workgroup, WM x WN wavefronts. Steps of 64 columns go
// through LDS, STAGES of them, all but one on their way from memory. x's rows are 64
// bytes of LDS; piece p of row r sits at p ^ f(r), so that the lanes of a fragment's
// read that go together are in different banks.
template <int BM, int BN, int WM, int WN, int STAGES>
__global__ __launch_bounds__(64 * WM * WN) void w8_kernel(W8Args a) {
  constexpr int WAVES = WM * WN;
  constexpr int AT = BM / 16 / WM, BT = BN / 16 / WN;        // tiles of a wavefront
  constexpr int AB = BM * 64, BB = BN * 64;                  // bytes of a stage
  constexpr int AL = AB / 1024 / WAVES, BL = BB / 1024 / WAVES, LOADS = AL + BL;
  static_assert(AL * WAVES * 1024 == AB && BL * WAVES * 1024 == BB, "whole loads for every wavefront");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[STAGES][AB + BB];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n16 = lane & 15, g = lane >> 4;
  const int wm = wave / WN, wn = wave % WN;
  // Workgroups go round the 8 XCDs: each XCD gets a run of tiles, in columns 8 high, so
  // that what runs there at a time shares rows of x and of the weights in its cache.
  const int total = a.mt * a.nt, per = (total + 7) / 8;
  const int t = (int)(blockIdx.x & 7) * per + (int)(blockIdx.x >> 3);
  if (t >= total || (int)(blockIdx.x >> 3) >= per) return;
  const int band = t / (8 * a.nt), high = min(8, a.mt - 8 * band), in_band = t - band * 8 * a.nt;
  const int bm = 8 * band + in_band % high, bn = in_band / high;
  const int64_t m0 = (int64_t)bm * BM;
  const int tile0 = bn * (BN / 16);

  const int rows = min((int64_t)BM, a.M - m0);
  const i32x4 rx = buffer_of(a.x + m0 * a.x_stride, (uint32_t)((rows - 1) * a.x_stride + (a.K + 15) / 16 * 16));   // (K, or rows laid out again)
  const int tiles = min(BN / 16, a.tiles - tile0);
  const i32x4 rw = buffer_of(a.codes + (size_t)tile0 * a.kblocks * 1024, (uint32_t)tiles * (uint32_t)a.kblocks * 1024u);
  const uint32_t base = (uint32_t)reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)&lds[0][0]);
  uint32_t xo[AL], wo[BL];
#pragma unroll
  for (int i = 0; i < AL; ++i) {
    const int row = 16 * (i * WAVES + wave) + (lane >> 2);
    const int f = (0x1230 >> (4 * ((row >> 2) & 3))) & 3;    // 0, 3, 2, 1
    xo[i] = row < rows ? (uint32_t)(row * a.x_stride + 16 * ((lane & 3) ^ f)) : kOutside;
  }
#pragma unroll
  for (int i = 0; i < BL; ++i) {
    const int tile = i * WAVES + wave;
    wo[i] = tile < tiles ? (uint32_t)tile * (uint32_t)a.kblocks * 1024u + 16 * lane : kOutside;
  }
  auto fetch = [&](int kb, int stage) {
    const bool in = kb < a.kblocks;   // (past the end nothing is read: the number of loads on their way stays the same)
    const uint32_t to = base + stage * (AB + BB);
#pragma unroll
    for (int i = 0; i < AL; ++i) load_lds(rx, in ? xo[i] + kb * 64 : kOutside, to + (i * WAVES + wave) * 1024);
#pragma unroll
    for (int i = 0; i < BL; ++i) load_lds(rw, in ? wo[i] + kb * 1024 : kOutside, to + AB + (i * WAVES + wave) * 1024);
  };
  i32x4 acc[BT][AT];
#pragma unroll
  for (int i = 0; i < BT; ++i)
#pragma unroll
    for (int m = 0; m < AT; ++m) acc[i][m] = i32x4{0, 0, 0, 0};
  const int f = (0x1230 >> (4 * ((n16 >> 2) & 3))) & 3;
  const uint32_t xr = (wm * AT * 16 + n16) * 64 + 16 * (g ^ f), wr = AB + wn * BT * 1024 + 16 * lane;
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) fetch(s, s);
  int stage = 0, ahead = STAGES - 1;
  for (int kb = 0; kb < a.kblocks; ++kb) {
    // this step's loads are done (those of the STAGES - 2 after it may not be), and every
    // wavefront has read the stage that is filled next
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"((STAGES - 2) * LOADS) : "memory");
    fetch(kb + STAGES - 1, ahead);
    const uint8_t* const from = lds[stage];
    i32x4 wf[BT], xf[AT];
#pragma unroll
    for (int i = 0; i < BT; ++i) wf[i] = *reinterpret_cast<const i32x4*>(from + wr + i * 1024);
#pragma unroll
    for (int m = 0; m < AT; ++m) xf[m] = *reinterpret_cast<const i32x4*>(from + xr + m * 1024);
#pragma unroll
    for (int m = 0; m < AT; ++m)
#pragma unroll
      for (int i = 0; i < BT; ++i) acc[i][m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[i], xf[m], acc[i][m], 0, 0, 0);
    stage = stage + 1 == STAGES ? 0 : stage + 1;
    ahead = ahead + 1 == STAGES ? 0 : ahead + 1;
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // (nothing may land in LDS after the workgroup's end)
#pragma unroll
  for (int i = 0; i < BT; ++i) {
    const int n = (tile0 + wn * BT + i) * 16 + 4 * g;
    float ws[4], b[4];
    load_four(a, n, ws, b);
#pragma unroll
    for (int m = 0; m < AT; ++m) {
      const int64_t row = m0 + (wm * AT + m) * 16 + n16;
      store_four(a, row, n, acc[i][m], row < a.M ? a.x_scale[row] : 0.f, ws, b);
    }
  }
}

// Rows of x that the large kernel cannot read 16 bytes at a time, laid out again.
__global__ __launch_bounds__(256) void w8_rows_kernel(const int8_t* x, int64_t x_stride, int64_t M, int32_t K, int32_t pieces, i32x4* out) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= M * pieces) return;
  const int64_t m = id / pieces;
  out[id] = row_piece(x + m * x_stride, (id - m * pieces) * 16, K);
}

struct W8Layout {
  int kblocks, tiles;
  size_t codes, total;
};

rsq_status w8_layout(int32_t n, int32_t k, W8Layout& l) {
  if (n < 1 || k < 1) return fail(RSQ_E_INVALID, "n %d k %d", n, k);
  // 2^17 products of -128 by -128 are 2^31, which int32 does not have
  if (k > (1 << 17) - 1) return fail(RSQ_E_UNSUPPORTED, "k %d: sums of 2^17 products and more leave int32", k);
  if (n > (1 << 26)) return fail(RSQ_E_UNSUPPORTED, "n %d above 2^26", n);
  l.kblocks = (k + 63) / 64;
  l.tiles = (n + 15) / 16;
  l.codes = (size_t)l.tiles * l.kblocks * 1024;
  l.total = l.codes + (size_t)n * 4;
  return RSQ_OK;
}

typedef void (*W8Fn)(W8Args);
struct W8Pick {
  W8Fn fn;
  int rows, tiles, waves;   // of a workgroup: rows of x, tiles of weight rows, wavefronts
  bool large;
};

// By the number of 16 x 16 tiles of y and the blocks of 64 columns, us (rows x n x k), the
// first shape taken:
//   to 600, long rows    two tiles, sixteen wavefronts: 64 x 2048 x 4096 5.3, four tiles and eight 6.4
//   to 1300              four tiles, eight wavefronts:  40 x 3000 x 1001 4.9, two and sixteen 6.1;
//                        16 x 12352 x 2048 5.2, blocks of 64 x 64 7.3
//   to 2600 (1800 where  32 rows of four tiles, four wavefronts: 256 x 2048 x 4096 8.9, blocks of 64 x 64
//   rows are short)      11.7; 333 x 1031 x 705 6.4, 10.0; 100 x 3700 x 1000 8.1, 8.8; 64 x 6400 x 2048
//                        9.5, 10.5; but 256 x 1600 x 1024 7.0, 6.0; 270 x 1500 x 96 4.3, 3.8. Of short rows
//                        above 1800: 333 x 1700 x 1024 7.7, 5.9; 256 x 2049 x 1025 13.4, 9.6; but 128 x 4096
//                        x 2048 8.6, 10.0
//   to 9000              blocks of 64 x 64:   128 x 12352 x 2048 10.3, of 64 x 128 11.9; 512 x 4096 x 4096 16.4, 18.3
//   above                blocks of 64 x 128:  256 x 12352 x 2048 15.0, of 64 x 64 18.2
// Before the last two come blocks of 128 x 256, three stages of 24 KB, two workgroups a compute
// unit, where there are 190 workgroups and more and rows of more than 1024: 4096 x 12352 x 2048 115,
// of 64 x 128 142, of 256 x 256 165; 512 x 12352 x 2048 25.3, 29.6, 43 (of 160 to 192 workgroups with
// rows of 2048 both take 26 to 28, within 2%); but 700 x 7000 x 1024 (168 workgroups) 15.9, 13.4 and
// 4096 x 28672 x 1024 238, 224 (y is most of it); and of 256 x 256 where rows are longer than 6144 and
// those blocks fill four fifths of the compute units' rounds: 4096 x 28672 x 8192 882, of 128 x 256
// 954; 512 x 28672 x 8192 117, 138; but 4096 x 8192 x 6144 197, 184.
W8Pick pick_w8(int64_t m, int tiles, int kblocks) {
  const int64_t mtiles = ceil_div(m, 16), work = mtiles * tiles;
  if (work <= 600 && kblocks > 32) return {w8_few_kernel<2, 1, 16>, 16, 2, 16, false};
  if (mtiles == 1 || work <= 1300) return {w8_few_kernel<4, 1, 8>, 16, 4, 8, false};
  if (work <= (kblocks > 32 ? 2600 : 1800)) return {w8_few_kernel<4, 2, 4>, 32, 4, 4, false};
  const int64_t large = ceil_div(m, 256) * ceil_div(tiles, 16), rounds = ceil_div(large, 256);
  if (kblocks > 96 && large * 5 >= rounds * 256 * 4) return {w8_kernel<256, 256, 2, 4, 4>, 256, 16, 8, true};
  if (kblocks > 16 && ceil_div(m, 128) * ceil_div(tiles, 16) >= 190) return {w8_kernel<128, 256, 2, 4, 3>, 128, 16, 8, true};
  if (work <= 9000) return {w8_kernel<64, 64, 2, 2, 4>, 64, 4, 4, true};
  return {w8_kernel<64, 128, 2, 2, 4>, 64, 8, 4, true};
}

constexpr int64_t kMaxStride = 1 << 22;   // 256 rows then end below 2^30

bool as_they_are(const rsq_w8* p) {
  return aligned(p->x, 16) && p->x_stride % 16 == 0 && p->k % 16 == 0 && p->x_stride <= kMaxStride;
}

rsq_status check_w8(const rsq_w8* p, W8Layout& l) {
  if (!p) return fail(RSQ_E_INVALID, "w8 is NULL");
  if (const rsq_status s = w8_layout(p->n, p->k, l)) return s;
  if (p->out_dtype != RSQ_F32 && p->out_dtype != RSQ_BF16) return fail(RSQ_E_INVALID, "out_dtype %d", p->out_dtype);
  if (p->m < 0) return fail(RSQ_E_INVALID, "m %d", p->m);
  if (p->m > 0 && (p->x_stride < p->k || p->y_stride < p->n)) return fail(RSQ_E_INVALID, "a row stride is shorter than its row");
  return RSQ_OK;
}

// bytes of the rows laid out again
size_t w8_rows_bytes(const rsq_w8* p, const W8Layout& l) {
  if (p->m == 0 || !pick_w8(p->m, l.tiles, l.kblocks).large || as_they_are(p)) return 0;
  return (size_t)p->m * ceil_div(p->k, 16) * 16;
}

}  // namespace
}  // namespace rsq

using namespace rsq;

extern "C" rsq_status rsq_w8_bytes(int32_t n, int32_t k, size_t* bytes) {
  if (!bytes) return fail(RSQ_E_INVALID, "bytes is NULL");
  W8Layout l;
  if (const rsq_status s = w8_layout(n, k, l)) return s;
  *bytes = l.total;
  return RSQ_OK;
}

extern "C" rsq_status rsq_w8_pack(const int8_t* codes, const float* scales, int32_t n, int32_t k, void* packed, size_t packed_bytes,
                                  void* stream) {
  W8Layout l;
  if (const rsq_status s = w8_layout(n, k, l)) return s;
  if (!codes || !scales || !packed) return fail(RSQ_E_INVALID, "codes, scales and packed must be non-NULL");
  if (!aligned(packed, 16) || !aligned(scales, 4)) return fail(RSQ_E_INVALID, "packed or scales is not aligned");
  if (packed_bytes < l.total) return fail(RSQ_E_BUFFER, "packed has %zu bytes, the weights need %zu", packed_bytes, l.total);
  const Span written[] = {{packed, (int64_t)l.total, "packed"}};
  const Span read[] = {{codes, (int64_t)n * k, "codes"}, {scales, (int64_t)n * 4, "scales"}};
  if (const rsq_status s = check_overlap(written, read)) return s;
  PackArgs a{codes, scales, static_cast<u32x2*>(packed), reinterpret_cast<float*>(static_cast<uint8_t*>(packed) + l.codes),
             n, k, l.kblocks, (int64_t)(l.codes / 16)};
  const int64_t blocks = ceil_div(a.pieces, 256);   // (16 pieces and more a tile of 16 rows: all scales are covered)
  if (const rsq_status s = check_blocks(blocks, 256)) return s;
  hipLaunchKernelGGL(w8_pack_kernel, dim3((unsigned)blocks), dim3(256), 0, (hipStream_t)stream, a);
  return launched("8-bit weight packing");
}

extern "C" rsq_status rsq_w8_workspace(const rsq_w8* p, size_t* bytes) {
  if (!bytes) return fail(RSQ_E_INVALID, "bytes is NULL");
  W8Layout l;
  if (const rsq_status s = check_w8(p, l)) return s;
  *bytes = w8_rows_bytes(p, l);
  return RSQ_OK;
}

extern "C" rsq_status rsq_w8_linear(const rsq_w8* p, void* stream) {
  W8Layout l;
  if (const rsq_status s = check_w8(p, l)) return s;
  if (p->m == 0) return RSQ_OK;   // (an empty tensor has no address)
  if (!p->x || !p->x_scale || !p->packed || !p->y) return fail(RSQ_E_INVALID, "x, x_scale, packed and y must be non-NULL");
  const int osize = p->out_dtype == RSQ_BF16 ? 2 : 4;
  if (!aligned(p->y, osize) || !aligned(p->x_scale, 4) || !aligned(p->bias, 4) || !aligned(p->packed, 16))
    return fail(RSQ_E_INVALID, "a pointer is not aligned to its element type (packed: 16 bytes)");
  if (p->packed_bytes < l.total)
    return fail(RSQ_E_BUFFER, "packed has %zu bytes, the weights need %zu", p->packed_bytes, l.total);
  const size_t again = w8_rows_bytes(p, l);
  if (again) {
    if (!p->workspace || !aligned(p->workspace, 16)) return fail(RSQ_E_INVALID, "workspace is NULL or not 16-byte aligned");
    if (p->workspace_bytes < again)
      return fail(RSQ_E_BUFFER, "workspace has %zu bytes, the product needs %zu", p->workspace_bytes, again);
  }
  const Span written[] = {{p->y, span_bytes(p->m, p->y_stride, p->n, osize), "y"},
                          {p->workspace, (int64_t)p->workspace_bytes, "workspace"}};
  const Span read[] = {{p->x, span_bytes(p->m, p->x_stride, p->k, 1), "x"},
                       {p->packed, (int64_t)l.total, "packed"},
                       {p->x_scale, (int64_t)p->m * 4, "x_scale"},
                       {p->bias, (int64_t)p->n * 4, "bias"}};
  if (const rsq_status s = check_overlap(written, read)) return s;
  W8Args a{};
  a.x = p->x, a.x_stride = p->x_stride;
  a.codes = static_cast<const uint8_t*>(p->packed);
  a.scale = reinterpret_cast<const float*>(a.codes + l.codes);
  a.x_scale = p->x_scale, a.bias = p->bias;
  a.y = p->y, a.y_stride = p->y_stride;
  a.M = p->m, a.N = p->n, a.K = p->k;
  a.kblocks = l.kblocks, a.tiles = l.tiles;
  a.out_bf16 = p->out_dtype == RSQ_BF16;
  a.wide = aligned(p->y, 4 * osize) && p->y_stride % 4 == 0;
  const W8Pick w = pick_w8(p->m, l.tiles, l.kblocks);
  a.mt = (int32_t)ceil_div(p->m, w.rows), a.nt = (int32_t)ceil_div(l.tiles, w.tiles);
  if (!w.large) {
    hipLaunchKernelGGL(w.fn, dim3((unsigned)a.nt, (unsigned)a.mt), dim3(64 * w.waves), 0, (hipStream_t)stream, a);
    return launched("8-bit product");
  }
  const int64_t blocks = ceil_div((int64_t)a.mt * a.nt, 8) * 8;
  if (const rsq_status s = check_blocks(blocks, 64 * w.waves)) return s;
  if (again) {
    const int64_t pieces = ceil_div(p->k, 16), copies = ceil_div(p->m * pieces, 256);
    if (const rsq_status s = check_blocks(copies, 256)) return s;
    hipLaunchKernelGGL(w8_rows_kernel, dim3((unsigned)copies), dim3(256), 0, (hipStream_t)stream, p->x, p->x_stride, (int64_t)p->m, p->k,
                       (int32_t)pieces, static_cast<i32x4*>(p->workspace));
    if (const rsq_status s = launched("8-bit product, rows")) return s;
    a.x = static_cast<const int8_t*>(p->workspace), a.x_stride = pieces * 16;
  }
  hipLaunchKernelGGL(w.fn, dim3((unsigned)blocks), dim3(64 * w.waves), 0, (hipStream_t)stream, a);
  return launched("8-bit product");
}

// Short causal convolution of every channel, before a selective scan:
//   y[t, c] = act(bias[c] + sum_{j < W} w[c, j] x[t - W + 1 + j, c]),  W = 2..4,
// act = silu or nothing. Inputs before a sequence's first come from its state
// [channels][W - 1] (oldest first; none: zeros), which takes the last W - 1
// inputs afterwards.
//
// A read and a write of every element against 2 W operations: bound by memory.
// A lane owns 16 bytes of consecutive channels, so that a wavefront reads 1 KB
// runs, and walks a tile of tokens with the last W - 1 inputs in registers; a tile
// reads W - 1 rows again (from L2). The next kAhead rows are loaded while the
// last ones are worked on, and kept as they come (bf16 pairs) until then: 16384 x
// 4352 bf16 (286 MB) 68 us, 4.2 TB/s, where a large copy moves 4.9; loaded one
// row at a time 98. 1531 x 1031 fp32, one element a lane, 6.0 us.
#include <type_traits>

#include "host_util.hpp"
#include "layer_ops.hpp"

namespace rsq {
namespace {

constexpr int kAhead = 4;   // rows loaded ahead
constexpr int kWaves = 4;   // wavefronts of a block, each with a tile of its own

struct ConvArgs {
  const void* x;
  void* y;
  void* state;
  const float* weight;
  const float* bias;
  int64_t x_stride, y_stride;
  Sequences q;
  int32_t C;
  int32_t cblocks, tiles;   // blocks along the channels; blocks along a sequence
  int32_t tile;             // tokens of a wavefront
  int32_t per, last;        // listed blocks: how many a workgroup takes, and the last workgroup along them
};

// exp(-v) saturates to infinity for v below about -88, and silu(v), there smaller
// than 2^-120, becomes -0. bf16 results take the hardware's exp2 and reciprocal (their errors, a few
// 2^-23, vanish in the rounding to 8 bits); fp32 ones the exact division.
template <typename T>
__device__ __forceinline__ float silu(float v) {
  if constexpr (std::is_same<T, float>::value) return v / (1.f + expf(-v));
  else return v * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(v * -1.44269504f));
}

template <typename T, int W, int VEC, bool SILU>
__device__ __forceinline__ void conv_out(const float (&win)[W][VEC], const float (&w)[VEC][W], const float (&b)[VEC],
                                         float (&out)[VEC]) {
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    float acc = b[e];
#pragma unroll
    for (int j = 0; j < W; ++j) acc = __builtin_fmaf(w[e][j], win[j][e], acc);
    out[e] = SILU ? silu<T>(acc) : acc;
  }
}

template <typename T, int VEC>
__device__ __forceinline__ void load_row(const T* p, float (&v)[VEC]) {
  if constexpr (VEC == 1) v[0] = to_f32(p[0]);
  else load_vec<VEC>(p, v);
}

// a row's VEC elements as loaded
template <typename T, int VEC>
struct RawRow {
  uint32_t w[VEC == 1 ? 1 : 4];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (VEC == 1) {
      w[0] = sizeof(T) == 2 ? *reinterpret_cast<const uint16_t*>(p) : *reinterpret_cast<const uint32_t*>(p);
    } else {
      const uint4 t = *reinterpret_cast<const uint4*>(p);
      w[0] = t.x, w[1] = t.y, w[2] = t.z, w[3] = t.w;
    }
  }
  __device__ __forceinline__ void get(float (&v)[VEC]) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] = __uint_as_float(w[e]);
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] = __uint_as_float((e & 1) ? w[e >> 1] & 0xFFFF0000u : w[e >> 1] << 16);
    }
  }
};

template <typename T, int VEC>
__device__ __forceinline__ void store_row(T* p, const float (&v)[VEC]) {
  if constexpr (VEC == 1) from_f32(v[0], p[0]);
  else store_vec<VEC>(p, v);
}

// weights of VEC channels ([channel][tap], so VEC * W consecutive floats) and their biases
template <int W, int VEC>
__device__ __forceinline__ void load_params(const ConvArgs& a, int c, float (&w)[VEC][W], float (&b)[VEC]) {
  if constexpr (VEC == 1) {
#pragma unroll
    for (int j = 0; j < W; ++j) w[0][j] = a.weight[(size_t)c * W + j];
    b[0] = a.bias ? a.bias[c] : 0.f;
  } else {
    float flat[VEC * W];
    load_vec<VEC * W>(a.weight + (size_t)c * W, flat);
#pragma unroll
    for (int e = 0; e < VEC; ++e)
#pragma unroll
      for (int j = 0; j < W; ++j) w[e][j] = flat[e * W + j];
    if (a.bias) load_vec<VEC>(a.bias + c, b);
    else
#pragma unroll
      for (int e = 0; e < VEC; ++e) b[e] = 0.f;
  }
}

// The state of VEC channels: VEC (W - 1) consecutive elements, h[j] the input
// W - 1 - j before the sequence.
template <typename T, int W, int VEC>
__device__ __forceinline__ void load_state(const T* p, float (&h)[W - 1][VEC]) {
  float flat[VEC * (W - 1)];
  if constexpr (VEC == 1) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) flat[j] = to_f32(p[j]);
  } else {
    load_vec<VEC*(W - 1)>(p, flat);
  }
#pragma unroll
  for (int e = 0; e < VEC; ++e)
#pragma unroll
    for (int j = 0; j < W - 1; ++j) h[j][e] = flat[e * (W - 1) + j];
}

template <typename T, int W, int VEC>
__device__ __forceinline__ void store_state(T* p, const float (&h)[W - 1][VEC]) {
  float flat[VEC * (W - 1)];
#pragma unroll
  for (int e = 0; e < VEC; ++e)
#pragma unroll
    for (int j = 0; j < W - 1; ++j) flat[e * (W - 1) + j] = h[j][e];
  if constexpr (VEC == 1) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) from_f32(flat[j], p[j]);
  } else {
    store_vec<VEC*(W - 1)>(p, flat);
  }
}

// One wavefront's tile of a sequence: channels c .. of tokens t0 ..
template <typename T, int W, int VEC, bool SILU>
__device__ __forceinline__ void conv_tile(const ConvArgs& a, int s, int64_t begin, int64_t len, int64_t t0, int c) {
  if (c >= a.C || t0 >= len) return;   // (an empty sequence keeps its state)
  const T* x = reinterpret_cast<const T*>(a.x) + begin * a.x_stride + c;
  T* y = reinterpret_cast<T*>(a.y) + begin * a.y_stride + c;
  T* st = a.state ? reinterpret_cast<T*>(a.state) + ((size_t)s * a.C + c) * (W - 1) : nullptr;
  float w[VEC][W], b[VEC];
  load_params<W, VEC>(a, c, w, b);
  float win[W][VEC];   // win[W - 1] is the current input
  auto before = [&](float (&h)[W - 1][VEC]) {
    if (st) load_state<T, W, VEC>(st, h);
    else
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
#pragma unroll
        for (int e = 0; e < VEC; ++e) h[j][e] = 0.f;
  };
  if (t0 == 0) {
    float old[W - 1][VEC];
    before(old);
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
#pragma unroll
      for (int e = 0; e < VEC; ++e) win[j][e] = old[j][e];
  } else {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) load_row<T, VEC>(x + (t0 - (W - 1) + j) * a.x_stride, win[j]);
  }
  const int n = (int)(len - t0 < a.tile ? len - t0 : a.tile);
  x += t0 * a.x_stride;
  y += t0 * a.y_stride;
  RawRow<T, VEC> rows[kAhead], next[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) next[i].load(x + (int64_t)(i < n ? i : n - 1) * a.x_stride);
  for (int i0 = 0; i0 < n; i0 += kAhead) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) rows[i] = next[i];
    if (i0 + kAhead < n) {
      // (past the last row, that row again)
#pragma unroll
      for (int i = 0; i < kAhead; ++i) next[i].load(x + (int64_t)(i0 + kAhead + i < n ? i0 + kAhead + i : n - 1) * a.x_stride);
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (i0 + i < n) {
        rows[i].get(win[W - 1]);
        float out[VEC];
        conv_out<T, W, VEC, SILU>(win, w, b, out);
        store_row<T, VEC>(y + (int64_t)(i0 + i) * a.y_stride, out);
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
#pragma unroll
          for (int e = 0; e < VEC; ++e) win[j][e] = win[j + 1][e];
      }
    }
  }
  // The lane of the first tile is the only reader of this state, and it writes
  // the new one. Inputs t < 0 are the old state's.
  if (t0 == 0 && st) {
    float old[W - 1][VEC];
    if (len < W - 1) before(old);
    float last[W - 1][VEC];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      const int64_t t = len - (W - 1) + j;
      if (t >= 0) {
        load_row<T, VEC>(x + t * a.x_stride, last[j]);   // (x is the sequence's first row: t0 = 0)
      } else {
        // t + W - 1 = len + j with 0 < len < W - 1
#pragma unroll
        for (int k = 0; k < W - 1; ++k)
          if (k == (int)(len + j))
#pragma unroll
            for (int e = 0; e < VEC; ++e) last[j][e] = old[k][e];
      }
    }
    store_state<T, W, VEC>(st, last);
  }
}

// A workgroup for every block of tokens (kWaves tiles) and of channels that the
// longest sequence has, in every sequence.
template <typename T, int W, int VEC, bool SILU>
__global__ __launch_bounds__(64 * kWaves) void conv_prompt_kernel(ConvArgs a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int64_t id = blockIdx.x;
  const int cb = (int)(id % a.cblocks);
  id /= a.cblocks;
  const int64_t tile = id % a.tiles;
  const int s = (int)(id / a.tiles);
  int64_t len;
  const int64_t begin = seq_range(a.q, s, len);
  conv_tile<T, W, VEC, SILU>(a, s, begin, len, (tile * kWaves + wave) * a.tile, (cb * 64 + lane) * VEC);
}

// sum over the lanes up to this one
__device__ __forceinline__ int wave_scan(int v, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(v, d, 64);
    if (lane >= d) v += o;
  }
  return v;
}

// Only the blocks that sequences have, listed sequence by sequence: `per` of them
// in a row for a workgroup, all that are left for the last one (where offsets fall
// there may be more than rows allow for). Wavefronts search the offsets for their first block, and
// for the next sequence with tokens, 64 sequences at a time.
template <typename T, int W, int VEC, bool SILU>
__global__ __launch_bounds__(64 * kWaves) void conv_list_kernel(ConvArgs a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int cb = (int)(blockIdx.x % a.cblocks), group = (int)(blockIdx.x / a.cblocks);
  const int rows = a.tile * kWaves;
  int64_t left = group == a.last ? INT64_MAX : a.per;
  int64_t skip = (int64_t)group * a.per;   // blocks before the wanted one, in sequences s0 and on
  int64_t s0 = 0;
  if (!a.q.offsets) s0 = skip / a.tiles, skip -= s0 * a.tiles;
  while (s0 < a.q.seqs) {
    int64_t begin = 0, len = 0;
    if (s0 + lane < a.q.seqs) begin = seq_range(a.q, (int)(s0 + lane), len);
    const int n = (int)((len + rows - 1) / rows);
    const int upto = wave_scan(n, lane);
    const uint64_t hit = __builtin_amdgcn_ballot_w64(skip < upto);
    if (!hit) {
      skip -= __builtin_amdgcn_readlane(upto, 63);
      s0 += 64;
      continue;
    }
    const int l = __builtin_ctzll(hit);
    const int mine = __builtin_amdgcn_readlane(n, l);
    const int64_t first = __builtin_amdgcn_readlane((int)begin, l), tokens = __builtin_amdgcn_readlane((int)len, l);
    for (int tile = (int)(skip - (__builtin_amdgcn_readlane(upto, l) - mine)); tile < mine; ++tile) {
      conv_tile<T, W, VEC, SILU>(a, (int)(s0 + l), first, tokens, ((int64_t)tile * kWaves + wave) * a.tile, (cb * 64 + lane) * VEC);
      if (--left == 0) return;
    }
    s0 += l + 1;
    skip = 0;
  }
}

// One token of every sequence: a lane per VEC channels of a sequence. The state
// (W - 1 inputs a channel, read and written) is most of the traffic. 128
// sequences of 4352 channels (9 MB) take 5.3 us, where an empty launch takes 4.6.
template <typename T, int W, int VEC, bool SILU>
__global__ __launch_bounds__(256) void conv_token_kernel(ConvArgs a) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int cv = (a.C + VEC - 1) / VEC;
  const int64_t s = id / cv;
  if (s >= a.q.seqs) return;
  const int c = (int)(id - s * cv) * VEC;
  T* st = a.state ? reinterpret_cast<T*>(a.state) + ((size_t)s * a.C + c) * (W - 1) : nullptr;
  float win[W][VEC], h[W - 1][VEC], w[VEC][W], b[VEC], out[VEC];
  load_row<T, VEC>(reinterpret_cast<const T*>(a.x) + s * a.x_stride + c, win[W - 1]);
  if (st) load_state<T, W, VEC>(st, h);
  else
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
#pragma unroll
      for (int e = 0; e < VEC; ++e) h[j][e] = 0.f;
  load_params<W, VEC>(a, c, w, b);
#pragma unroll
  for (int j = 0; j < W - 1; ++j)
#pragma unroll
    for (int e = 0; e < VEC; ++e) win[j][e] = h[j][e];
  conv_out<T, W, VEC, SILU>(win, w, b, out);
  store_row<T, VEC>(reinterpret_cast<T*>(a.y) + s * a.y_stride + c, out);
  if (st) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
#pragma unroll
      for (int e = 0; e < VEC; ++e) h[j][e] = win[j + 1][e];
    store_state<T, W, VEC>(st, h);
  }
}

typedef void (*ConvFn)(ConvArgs);

enum ConvForm { kToken, kBlocks, kList };

template <typename T, int W, int VEC>
ConvFn pick(ConvForm form, bool silu) {
  if (form == kToken) return silu ? conv_token_kernel<T, W, VEC, true> : conv_token_kernel<T, W, VEC, false>;
  if (form == kList) return silu ? conv_list_kernel<T, W, VEC, true> : conv_list_kernel<T, W, VEC, false>;
  return silu ? conv_prompt_kernel<T, W, VEC, true> : conv_prompt_kernel<T, W, VEC, false>;
}

template <typename T, int VEC>
ConvFn pick_width(int width, ConvForm form, bool silu) {
  switch (width) {
    case 2: return pick<T, 2, VEC>(form, silu);
    case 3: return pick<T, 3, VEC>(form, silu);
    default: return pick<T, 4, VEC>(form, silu);
  }
}

}  // namespace
}  // namespace rsq

using namespace rsq;

extern "C" rsq_status rsq_causal_conv(const rsq_conv* p, void* stream) {
  if (!p) return fail(RSQ_E_INVALID, "conv is NULL");
  if (p->dtype != RSQ_F32 && p->dtype != RSQ_BF16) return fail(RSQ_E_INVALID, "dtype %d", p->dtype);
  if (p->activation != RSQ_ACT_NONE && p->activation != RSQ_ACT_SILU)
    return fail(RSQ_E_INVALID, "activation %d", p->activation);
  if (p->seqs < 1 || p->channels < 1) return fail(RSQ_E_INVALID, "seqs %d channels %d", p->seqs, p->channels);
  if (p->width < 2 || p->width > 4) return fail(RSQ_E_UNSUPPORTED, "width %d not in 2..4", p->width);
  if (p->tokens < 0 || p->tokens > 0x7fffffff) return fail(RSQ_E_INVALID, "tokens %lld", (long long)p->tokens);
  if (p->max_len < 0 || p->max_len > p->tokens) return fail(RSQ_E_INVALID, "max_len %lld of %lld tokens",
                                                            (long long)p->max_len, (long long)p->tokens);
  if (!p->offsets && p->tokens != p->max_len * p->seqs)
    return fail(RSQ_E_INVALID, "without offsets every sequence has max_len rows: %lld tokens, %d of %lld",
                (long long)p->tokens, p->seqs, (long long)p->max_len);
  if (p->max_len == 0) return RSQ_OK;
  if (!p->x || !p->weight || !p->y) return fail(RSQ_E_INVALID, "x, weight and y must be non-NULL");
  if (p->x_stride < p->channels || p->y_stride < p->channels)
    return fail(RSQ_E_INVALID, "row strides %lld, %lld below %d channels", (long long)p->x_stride,
                (long long)p->y_stride, p->channels);
  const int size = p->dtype == RSQ_BF16 ? 2 : 4;
  if (!aligned(p->x, size) || !aligned(p->y, size) || !aligned(p->state, size) || !aligned(p->weight, 4) ||
      !aligned(p->bias, 4) || !aligned(p->offsets, 4))
    return fail(RSQ_E_INVALID, "a pointer is not aligned to its element type");
  const int64_t C = p->channels;
  const Span written[] = {{p->y, span_bytes(p->tokens, p->y_stride, C, size), "y"},
                          {p->state, (int64_t)p->seqs * C * (p->width - 1) * size, "state"}};
  const Span read[] = {{p->x, span_bytes(p->tokens, p->x_stride, C, size), "x"},
                       {p->weight, C * p->width * 4, "weight"},
                       {p->bias, C * 4, "bias"},
                       {p->offsets, ((int64_t)p->seqs + 1) * 4, "offsets"}};
  if (const rsq_status s = check_overlap(written, read)) return s;

  // 16-byte accesses where every row, parameter and state address allows them
  // (one prompt of 16384 x 4352 bf16 63 us), one element at a time otherwise, at
  // any alignment (70)
  const int vec = 16 / size;
  const bool wide = C % vec == 0 && p->x_stride % vec == 0 && p->y_stride % vec == 0 && aligned(p->x, 16) &&
                    aligned(p->y, 16) && aligned(p->state, 16) && aligned(p->weight, 16) && aligned(p->bias, 16);
  const int v = wide ? vec : 1;
  const bool token = !p->offsets && p->max_len == 1, silu = p->activation == RSQ_ACT_SILU;
  ConvArgs a{};
  a.x = p->x, a.y = p->y, a.state = p->state, a.weight = p->weight, a.bias = p->bias;
  a.x_stride = p->x_stride, a.y_stride = p->y_stride;
  a.q = Sequences{p->offsets, p->tokens, p->max_len, p->seqs};
  a.C = p->channels;
  a.cblocks = (int32_t)ceil_div(C, 64 * v);
  // Tiles of 32 tokens re-read 3 rows of 35; where they leave the chip short of
  // wavefronts (16 for each of 256 compute units), shorter ones wait less: 1531 x
  // 1031 fp32 one element a lane 9.6 us with 32, 6.9 with 8.
  a.tile = 32;
  while (a.tile > 8 && a.cblocks * ceil_div(p->tokens, a.tile) < 4096) a.tile /= 2;
  a.tiles = (int32_t)ceil_div(p->max_len, (int64_t)a.tile * kWaves);
  const int64_t blocks = (int64_t)a.cblocks * a.tiles * p->seqs;
  // Of packed sequences with their rows apart, at most `listed` blocks have tokens.
  // A workgroup without any costs 0.8 ns, finding the others' blocks about 1 ns each
  // for every 64 sequences that are searched. us with blocks of all sequences and
  // with listed ones, 16384 x 4352 bf16: 8 sequences, 2.8 times the listed blocks 67
  // and 69, 4.2 times 62 and 59; 16345 tokens among 39 of one 82 and 59; 16384 beside
  // 255 of one 276 and 70. 65536 tokens with one of 60000 among 1024 sequences 3430
  // and 339; 1024 equal ones of 64 (1024 channels) 58 and 101.
  const int64_t rows = (int64_t)a.tile * kWaves, listed = p->offsets ? p->tokens / rows + p->seqs : (int64_t)a.tiles * p->seqs;
  const bool list = !token && (blocks > max_blocks(64 * kWaves) || blocks > 4 * listed * a.cblocks);
  const ConvForm form = token ? kToken : list ? kList : kBlocks;
  ConvFn fn;
  if (p->dtype == RSQ_BF16) fn = wide ? pick_width<Bf16, 8>(p->width, form, silu) : pick_width<Bf16, 1>(p->width, form, silu);
  else fn = wide ? pick_width<float, 4>(p->width, form, silu) : pick_width<float, 1>(p->width, form, silu);
  if (list) {
    // (more in a row where each search is long; one of 20000 tokens among 20000 short ones 2152 us, one by one 35000)
    a.per = (int32_t)(1 + p->seqs / 256 + listed * a.cblocks / max_blocks(64 * kWaves));
    const int64_t groups = ceil_div(listed, a.per);
    a.last = (int32_t)(groups - 1);
    if (const rsq_status s = check_blocks(groups * a.cblocks, 64 * kWaves)) return s;
    hipLaunchKernelGGL(fn, dim3((unsigned)(groups * a.cblocks)), dim3(64 * kWaves), 0, (hipStream_t)stream, a);
    return launched("causal convolution, listed blocks");
  }
  if (!token) {
    hipLaunchKernelGGL(fn, dim3((unsigned)blocks), dim3(64 * kWaves), 0, (hipStream_t)stream, a);
    return launched("causal convolution");
  }
  // sequences beyond what one launch may have go into further ones
  const int64_t cv = ceil_div(C, v), most = max_blocks(256) * 256 / cv;
  for (int64_t done = 0; done < p->seqs; done += most) {
    a.q.seqs = (int32_t)(p->seqs - done < most ? p->seqs - done : most);
    a.x = static_cast<const uint8_t*>(p->x) + done * p->x_stride * size;
    a.y = static_cast<uint8_t*>(p->y) + done * p->y_stride * size;
    if (p->state) a.state = static_cast<uint8_t*>(p->state) + done * C * (p->width - 1) * size;
    hipLaunchKernelGGL(fn, dim3((unsigned)ceil_div(a.q.seqs * cv, 256)), dim3(256), 0, (hipStream_t)stream, a);
    if (const rsq_status s = launched("causal convolution, one token")) return s;
  }
  return RSQ_OK;
}

// Attention with the delta rule over prompts (linear.hpp has the recurrence), in
// chunks of kL tokens. With c_t the sum of log a over a chunk's tokens up to t, S0
// the state before the chunk and n its last token, the chunk's u solve
//   u_t + sum_{s < t} A_ts u_s = b_t (v_t - e^{c_t} S0^T k_t),  A_ts = b_t e^{c_t - c_s} (k_t . k_s),
// so that with T = (1 + A)^-1 diag(b), which does not depend on the state,
//   X = V - e^c K S0,   U = T X,
//   O = e^c Q S0 + P U,   P_ts = e^{c_t - c_s} (q_t . k_s) for s <= t,
//   S <- e^{c_n} S0 + K^T (e^{c_n - c} U).
// delta_prepare_kernel makes T and P of all chunks side by side; delta_kernel then
// follows the state through a sequence's chunks.
//
// 16384 tokens of 32 heads of 128 x 128 with 16 key heads (bf16, 411 MB, 60 GFLOP of the
// recurrence's own operations: 80 us) take 520 to 540 us (by the card): 87 for the chunks, which is memory (32 KB
// read, 25 written a chunk and head, 5.4 TB/s), and 436 for the chain of 256 chunks. A chunk of it
// takes 1.7 us, three steps of about 1150 cycles: in the first the state's pieces come
// through LDS (64 KB for eight wavefronts), in the second the products with T, in the third
// the state's update and its splitting into pieces, each step with an LDS round trip and a
// barrier; the products themselves are 800 cycles of a SIMD. A compute unit alone takes no
// less with fewer loads than 1.3 us; with all 256 busy, the 57 KB a chunk that each workgroup
// reads from its XCD's cache are the other limit. Measured without gain: K and Q copied
// into whole rows by the first kernel, the next chunk but one called into the cache ahead,
// raised priority for the wavefronts that make U, T's pieces stored as such (511 -> 566:
// more to read), a wavefront for 16 columns and all rows (no exchange, but 182 products and
// 800 vector instructions one after another: 1.1 ms), parts of K S0 summed through LDS (744 us).
// States keep 1.3e-7 to 1.5e-7 of their norm; two pieces instead of three would leave 2.4e-6.
#include <algorithm>

#include "chunk.hpp"
#include "host_util.hpp"
#include "linear.hpp"

namespace rsq {
namespace {

constexpr int kL = 64;       // tokens of a chunk
constexpr int kTiles = kL / 16;
constexpr int kPieces = 3;   // of fp32 factors that reach the state
typedef ChunkRows<kL> Rows;

struct DeltaArgs {
  LinearArgs l;
  uint8_t* chunks;    // [slot][head] what a chunk's tokens give (Chunk)
  uint8_t* keys;      // fp32: [slot][key head][K, Q][pieces][kL][DK] bf16
  int32_t vblocks;    // column blocks of a head
  int32_t units;      // sequences x heads
};

// What the first kernel leaves of a chunk and head for the second: fragments of T (fp32,
// to be split where there is time) and P^T (pieces) as products of 32 tokens s take
// them, those with an s <= t only, and the decays.
template <int PY>
struct Chunk {
  static constexpr int kFragments = 6;
  // fragment of tokens t in tile e, s in the j-th 32
  static __device__ constexpr int fragment(int e, int j) { return e < 2 ? e : 2 * e - 2 + j; }
  static constexpr int kT = 0, kP = kFragments * 2048, kGates = kP + kFragments * PY * 1024;
  static constexpr int kBytes = kGates + 1024;
  // bytes of the gates: e^{c_t}, e^{c_n - c_t}; then e^{c_n}; the first token whose key or gate is not finite
  static constexpr int kTo = kGates, kFrom = kTo + 4 * kL, kDecay = kFrom + 4 * kL, kBad = kDecay + 4;
};

// Chunk j of a sequence that begins at row b is slot b / kL + s + j: those of the
// sequences before it end below that, whatever their lengths.
__device__ __forceinline__ int first_slot(const Sequences& q, int s, int& begin, int& len) {
  int64_t n;
  begin = (int)seq_range(q, s, n);
  len = (int)n;
  return begin / kL + s;
}

// The sequence of a slot: the last one whose first slot is not above it. 64 sequences
// are looked at at a time, a 64th of those left apart.
__device__ __forceinline__ bool find_chunk(const Sequences& q, int slot, int lane, int& sq, int& begin, int& len, int& chunk) {
  int lo = 0, n = q.seqs;
  for (;;) {
    const int step = (n + 63) / 64, s = lo + lane * step;
    int b = 0, l = 0;
    const bool below = lane * step < n && first_slot(q, s, b, l) <= slot;
    const uint64_t hit = __builtin_amdgcn_ballot_w64(below);
    if (!hit) return false;
    const int last = 63 - __builtin_clzll(hit);
    if (step == 1) {
      begin = __builtin_amdgcn_readlane(b, last), len = __builtin_amdgcn_readlane(l, last);
      sq = lo + last;
      chunk = slot - (begin / kL + sq);
      return chunk * kL < len;
    }
    n = min(step, n - last * step);
    lo += last * step;
  }
}

// Three pieces of factors that reach the state, two of those that reach bf16 outputs only
__device__ __forceinline__ void split(float a, float b, uint32_t (&p)[3]) { split_even(a, b, p); }
__device__ __forceinline__ void split(float a, float b, uint32_t (&p)[2]) { split_pair<2>(a, b, p); }

__device__ __forceinline__ float exp2_of(double c) { return __builtin_amdgcn_exp2f((float)c); }

// A sequence of up to kFew tokens (a decode batch's beside a prompt, a few drafted ones), token
// by token with 64 columns of its state in registers, as the single-token form does: a chunk's
// work for each would be ten times what the state's bytes take. A wavefront owns 16 columns, a
// lane four of them and a 16th of the rows, so that no token waits for another wavefront. us so,
// and as chunks (32 heads of 128 x 128 bf16): 256 sequences of one token 237, 863 (1080 MB, 4.6
// TB/s), of eight 340, 875; one sequence of one 5.6, 14.4, of eight 10.8, 14.7; 255 of one beside
// one of 16384 750, 1396; 64 of eight beside one of 64 92, 209, but one of eight beside it 20, 17.
constexpr int kFew = 8;
template <int DK>
struct Few {
  float k[kFew][DK], q[kFew][DK], v[kFew][64];
  float alpha[kFew], beta[kFew];
  int bad;   // the first token whose key or gates are not finite: NaN from there on
};
// the sum of 16 neighbouring lanes, the same in each
__device__ __forceinline__ float sum16(float v) {
  v += __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), 0x128, 0xf, 0xf, false));
  v += __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), 0x124, 0xf, 0xf, false));
  v += __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), 0x122, 0xf, 0xf, false));
  v += __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(0, (int)__float_as_uint(v), 0x121, 0xf, 0xf, false));
  return v;
}
template <typename T, int DK>
__device__ __forceinline__ void few_tokens(const LinearArgs& l, Few<DK>& f, int sq, int h, int64_t begin, int len) {
  constexpr int NR = DK / 16;
  const int tid = threadIdx.x, c = 4 * (tid >> 4), r0 = (tid & 15) * NR;
  const int dk = l.dk, dv = l.dv, hk = h / l.per_key;
  const T* const k = reinterpret_cast<const T*>(l.k) + begin * l.k_stride + (int64_t)hk * dk;
  const T* const q = reinterpret_cast<const T*>(l.q) + begin * l.q_stride + (int64_t)hk * dk;
  const T* const v = reinterpret_cast<const T*>(l.v) + begin * l.v_stride + (int64_t)h * dv;
  T* const o = reinterpret_cast<T*>(l.o) + begin * l.o_stride + (int64_t)h * dv;
  float* const S = l.state + ((size_t)sq * l.H + h) * dk * dv;
  if (tid == 0) f.bad = kFew;
  __syncthreads();
  for (int e = tid; e < len * DK; e += 256) {
    const int t = e / DK, r = e % DK;
    const float kv = r < dk ? to_f32(k[t * l.k_stride + r]) : 0.f;
    f.k[t][r] = kv;
    f.q[t][r] = r < dk ? to_f32(q[t * l.q_stride + r]) : 0.f;
    if (!(fabsf(kv) < __builtin_inff())) atomicMin(&f.bad, t);
  }
  if (tid < len) {
    const float al = l.alpha ? l.alpha[(begin + tid) * l.alpha_stride + h] : 1.f, be = l.beta[(begin + tid) * l.beta_stride + h];
    f.alpha[tid] = al, f.beta[tid] = be;
    if (!(al >= 0.f && al < __builtin_inff() && fabsf(be) < __builtin_inff())) atomicMin(&f.bad, tid);
  }
  for (int v0 = 64 * blockIdx.y; v0 < dv; v0 += 64 * gridDim.y) {
    const bool in = v0 + c < dv;   // (d_v is a multiple of 4)
    float4 m[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i)
      m[i] = l.state_in && in && r0 + i < dk ? *reinterpret_cast<const float4*>(S + (size_t)(r0 + i) * dv + v0 + c)
                                             : make_float4(0.f, 0.f, 0.f, 0.f);
    for (int e = tid; e < len * 64; e += 256) {
      const int t = e >> 6, j = e & 63;
      f.v[t][j] = v0 + j < dv ? to_f32(v[t * l.v_stride + v0 + j]) : 0.f;
    }
    __syncthreads();
    // a token's factors are read while the one before is worked on
    f32x4 kn[NR / 4], qn[NR / 4], vn;
    float decay, beta;
    auto read = [&](int t) {
#pragma unroll
      for (int i = 0; i < NR / 4; ++i) {
        kn[i] = *reinterpret_cast<const f32x4*>(&f.k[t][r0 + 4 * i]);
        qn[i] = *reinterpret_cast<const f32x4*>(&f.q[t][r0 + 4 * i]);
      }
      vn = *reinterpret_cast<const f32x4*>(&f.v[t][c]);
      decay = f.alpha[t], beta = f.beta[t];
    };
    const int bad = f.bad;
    read(0);
    for (int t = 0; t < len; ++t) {
      float ks[4] = {0.f, 0.f, 0.f, 0.f}, qs[4] = {0.f, 0.f, 0.f, 0.f}, qk = 0.f;
      float kf[NR];
      const f32x4 vt = vn;
      const float strength = beta;
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        float* const p = &m[i].x;
        kf[i] = kn[i / 4][i % 4];
        const float qf = qn[i / 4][i % 4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          p[e] *= decay;
          ks[e] = __builtin_fmaf(kf[i], p[e], ks[e]);
          qs[e] = __builtin_fmaf(qf, p[e], qs[e]);
        }
        qk = __builtin_fmaf(kf[i], qf, qk);
      }
      read(min(t + 1, len - 1));
      qk = sum16(qk);
      float u[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x = vt[e] - sum16(ks[e]);
        u[e] = t < bad && fabsf(x) < __builtin_inff() ? strength * x : __builtin_nanf("");
        qs[e] = sum16(qs[e]);
      }
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        float* const p = &m[i].x;
#pragma unroll
        for (int e = 0; e < 4; ++e) p[e] = __builtin_fmaf(kf[i], u[e], p[e]);
      }
      if (r0 == 0 && in) {
#pragma unroll
        for (int e = 0; e < 4; ++e) from_f32(__builtin_fmaf(qk, u[e], qs[e]), o[t * l.o_stride + v0 + c + e]);
      }
    }
#pragma unroll
    for (int i = 0; i < NR; ++i)
      if (in && r0 + i < dk) *reinterpret_cast<float4*>(S + (size_t)(r0 + i) * dv + v0 + c) = m[i];
    __syncthreads();   // v has been read
  }
}

// One chunk of one head. K K^T and Q K^T on the matrix cores (exact products of the
// inputs' pieces); the inverse in fp32: 16 x 16 blocks on the diagonal by
// substitution, a column a lane, then the blocks below them, diagonal by diagonal,
// T_ij = -T_ii sum_k A_ik T_kj, by fp32 products.
template <typename T, int DK, int PI, int PY>
__global__ __launch_bounds__(256) void delta_prepare_kernel(DeltaArgs a) {
  typedef Tile<DK> TB;
  typedef Chunk<PY> C;
  constexpr int KS = DK / 32, LD = kL + 4;
  constexpr int BB = kL * TB::kBytes;
  constexpr int KEYS = 2 * PI * BB, INV = 2 * kL * LD * 4;
  // K and Q, and once their products are there, A and its inverse
  __shared__ __attribute__((aligned(16))) uint8_t raw[KEYS > INV ? KEYS : INV];
  // e^{c_t - c_s} of the chunk's tokens as products: c = n + f in powers of two with n whole,
  // 2^{f_t} 2^{-f_s} 2^{n_t - n_s}
  __shared__ __attribute__((aligned(16))) float lds_to[kL], lds_from[kL], lds_beta[kL];
  __shared__ __attribute__((aligned(16))) int lds_whole[kL];
  __shared__ int lds_bad;
  uint8_t* const lds_k = raw;
  uint8_t* const lds_q = raw + PI * BB;
  float* const lds_a = reinterpret_cast<float*>(raw);
  float* const lds_t = lds_a + kL * LD;

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n16 = lane & 15, g = lane >> 4;
  const int h = blockIdx.x % a.l.H;
  const int slot = blockIdx.x / a.l.H;
  int sq, begin, len, chunk;
  if (!find_chunk(a.l.s, slot, lane, sq, begin, len, chunk)) return;
  begin = __builtin_amdgcn_readfirstlane(begin), len = __builtin_amdgcn_readfirstlane(len);
  static_assert(sizeof(Few<DK>) <= sizeof(raw), "a few tokens fit where a chunk's keys do");
  if (len <= kFew) {
    few_tokens<T, DK>(a.l, *reinterpret_cast<Few<DK>*>(raw), sq, h, begin, len);
    return;
  }
  if (blockIdx.y > 0) return;
  const int t0 = __builtin_amdgcn_readfirstlane(chunk) * kL;
  const int hk = h / a.l.per_key, dk = a.l.dk;
  uint8_t* const blob = a.chunks + ((size_t)slot * a.l.H + h) * C::kBytes;

  // ---- rows to LDS
  constexpr int NB = kL * (DK / 8) / 256, RB = 256 / (DK / 8);
  const int row0 = tid / (DK / 8), piece = tid % (DK / 8);
  const int krow = (int)(a.l.k_stride * sizeof(T)), qrow = (int)(a.l.q_stride * sizeof(T));
  Vec8<T, PI> rk[NB], rq[NB];
  {
    const Rows rK(reinterpret_cast<const T*>(a.l.k) + begin * a.l.k_stride + (size_t)hk * dk, krow, t0, len);
    const Rows rQ(reinterpret_cast<const T*>(a.l.q) + begin * a.l.q_stride + (size_t)hk * dk, qrow, t0, len);
    const bool in = piece * 8 < dk;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      rk[i].load(rK, in ? (uint32_t)((row0 + i * RB) * krow + piece * 8 * (int)sizeof(T)) : kOutside);
      rq[i].load(rQ, in ? (uint32_t)((row0 + i * RB) * qrow + piece * 8 * (int)sizeof(T)) : kOutside);
    }
  }
  const bool valid = lane < kL && t0 + lane < len;
  float al = 1.f, be = 0.f;
  if (wave == 0 && valid) {
    const int64_t row = (int64_t)begin + t0 + lane;
    if (a.l.alpha) al = a.l.alpha[row * a.l.alpha_stride + h];
    be = a.l.beta[row * a.l.beta_stride + h];
  }
  if (tid == 0) lds_bad = kL;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int row = row0 + i * RB;
    const uint32_t at = TB::at(row, piece);
    u32x4 pk[PI], pq[PI];
    rk[i].template pieces<true>(pk);
    rq[i].template pieces<true>(pq);
#pragma unroll
    for (int p = 0; p < PI; ++p) {
      *reinterpret_cast<u32x4*>(lds_k + p * BB + at) = pk[p];
      *reinterpret_cast<u32x4*>(lds_q + p * BB + at) = pq[p];
    }
    if (rk[i].bad_bits() & (PI == 1 ? 0x80008000u : 0x80000000u)) atomicMin(&lds_bad, row);
    if constexpr (PI > 1) {
      if (h % a.l.per_key == 0) {
        uint8_t* const to = a.keys + ((size_t)slot * (a.l.H / a.l.per_key) + hk) * KEYS + row * TB::kBytes + piece * 16;
#pragma unroll
        for (int p = 0; p < PI; ++p) {
          *reinterpret_cast<u32x4*>(to + p * BB) = pk[p];
          *reinterpret_cast<u32x4*>(to + (PI + p) * BB) = pq[p];
        }
      }
    }
  }
  __syncthreads();
  // ---- decays. From a token on whose key or gates are not finite the whole state is
  // NaN: such tokens are left out here, and written as NaN by the second kernel.
  if (wave == 0) {
    const uint64_t odd = __builtin_amdgcn_ballot_w64(valid && !(al >= 0.f && al < __builtin_inff() && fabsf(be) < __builtin_inff()));
    const int bad = min(lds_bad, odd ? (int)__builtin_ctzll(odd) : kL);
    const bool in = valid && lane < bad;
    double cum = in ? log2((double)al) : 0.;
    cum = cum < -2000. ? -2000. : cum;   // (as good as nothing of an fp32 state is left)
    cum = wave_scan(cum);
    const double last = lane63(cum);
    const double whole = rint(cum);
    const float f = (float)(cum - whole);
    lds_to[lane] = __builtin_amdgcn_exp2f(f);
    lds_from[lane] = __builtin_amdgcn_exp2f(-f);
    lds_whole[lane] = (int)whole;
    lds_beta[lane] = in ? be : 0.f;
    *reinterpret_cast<float*>(blob + C::kTo + 4 * lane) = exp2_of(cum);
    *reinterpret_cast<float*>(blob + C::kFrom + 4 * lane) = exp2_of(last - cum);
    if (lane == 0) {
      *reinterpret_cast<float*>(blob + C::kDecay) = exp2_of(last);
      *reinterpret_cast<int*>(blob + C::kBad) = bad;
      lds_bad = bad;
    }
  }
  __syncthreads();
  const int bad = lds_bad;
  // ---- rows s, columns t, of the products with K (for A) and with Q (P^T): two tiles
  // of s at a time, a step of the products that take P
  const uint32_t a_frag = TB::fragment(lane);
  auto products = [&](int e, bool keys, f32x4 (&acc)[kL / 32][2]) {
    const uint8_t* const cols = keys ? lds_k : lds_q;
    const int t = 16 * e + n16;
    const float to = keys ? lds_to[t] * lds_beta[t] : lds_to[t];
    const int whole = lds_whole[t];
    u32x4 cf[KS][PI];
#pragma unroll
    for (int i = 0; i < KS; ++i)
#pragma unroll
      for (int p = 0; p < PI; ++p) cf[i][p] = *reinterpret_cast<const u32x4*>(cols + p * BB + 16 * e * TB::kBytes + (a_frag ^ (i << 6)));
#pragma unroll
    for (int j = 0; j < kL / 32; ++j) {
      acc[j][0] = acc[j][1] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (2 * j > e) continue;
#pragma unroll
      for (int i = 0; i < KS; ++i)
#pragma unroll
        for (int p = 0; p < PI; ++p)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const u32x4 kf = *reinterpret_cast<const u32x4*>(lds_k + p * BB + (32 * j + 16 * u) * TB::kBytes + (a_frag ^ (i << 6)));
#pragma unroll
            for (int q = 0; q < PI; ++q)
              if (p + q < 3) acc[j][u] = mfma(kf, cf[i][q], acc[j][u]);
          }
      settle();
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int s0 = 32 * j + 16 * u + 4 * g;
        const f32x4 from = *reinterpret_cast<const f32x4*>(&lds_from[s0]);
        const i32x4 n = *reinterpret_cast<const i32x4*>(&lds_whole[s0]);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float w = __builtin_amdgcn_ldexpf(acc[j][u][r] * (to * from[r]), whole - n[r]);
          // later tokens, and those from a bad one on, have no part whatever their products are
          acc[j][u][r] = s0 + r < bad && (keys ? s0 + r < t && t < bad : s0 + r <= t) ? w : 0.f;
        }
      }
    }
  };
  {
    const int e = 3 - wave;
    f32x4 p[kL / 32][2];
    products(e, false, p);
#pragma unroll
    for (int j = 0; j < kL / 32; ++j) {
      if (2 * j > e) continue;
      u32x4 pf[PY];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t lo[PY], hi[PY];
        split(p[j][u][0], p[j][u][1], lo);
        split(p[j][u][2], p[j][u][3], hi);
#pragma unroll
        for (int q = 0; q < PY; ++q) pf[q][2 * u] = lo[q], pf[q][2 * u + 1] = hi[q];
      }
#pragma unroll
      for (int q = 0; q < PY; ++q)
        *reinterpret_cast<u32x4*>(blob + C::kP + ((C::fragment(e, j) * PY + q) * 64 + lane) * 16) = pf[q];
    }
  }
  f32x4 kk[kL / 32][2];
  products(wave, true, kk);
  __syncthreads();   // K and Q have been read: A and its inverse take their place
#pragma unroll
  for (int j = 0; j < kL / 32; ++j)
#pragma unroll
    for (int u = 0; u < 2; ++u) *reinterpret_cast<f32x4*>(&lds_a[(16 * wave + n16) * LD + 32 * j + 16 * u + 4 * g]) = kk[j][u];
  __syncthreads();
  if (lane < 16) {
    float x[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float v = lane == i ? 1.f : 0.f;
#pragma unroll
      for (int m = 0; m < i; ++m) v = __builtin_fmaf(-lds_a[(16 * wave + i) * LD + 16 * wave + m], x[m], v);
      x[i] = v;
      lds_t[(16 * wave + i) * LD + 16 * wave + lane] = v;
    }
  }
  __syncthreads();
#pragma unroll
  for (int d = 1; d < kTiles; ++d) {
    if (wave < kTiles - d) {
      const int j = wave, i = wave + d;
      f32x4 m = {0.f, 0.f, 0.f, 0.f}, y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int k = 0; k < d; ++k)
#pragma unroll
        for (int st = 0; st < 4; ++st)
          m = __builtin_amdgcn_mfma_f32_16x16x4f32(lds_a[(16 * i + n16) * LD + 16 * (j + k) + 4 * st + g],
                                                   lds_t[(16 * (j + k) + 4 * st + g) * LD + 16 * j + n16], m, 0, 0, 0);
      settle();
      // a lane's sums are rows 4 g + r: one r at a time they are the next product's
#pragma unroll
      for (int r = 0; r < 4; ++r)
        y = __builtin_amdgcn_mfma_f32_16x16x4f32(lds_t[(16 * i + n16) * LD + 16 * i + 4 * g + r], m[r], y, 0, 0, 0);
      settle();
#pragma unroll
      for (int r = 0; r < 4; ++r) lds_t[(16 * i + 4 * g + r) * LD + 16 * j + n16] = -y[r];
    }
    __syncthreads();
  }
#pragma unroll
  for (int e = 0; e < kTiles; ++e)
#pragma unroll
    for (int j = 0; j <= e / 2; ++j) {
      const int f = C::fragment(e, j);
      if (f % 4 != wave) continue;
      const int t = 16 * e + n16;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        if (2 * j + u > e) continue;   // (nothing there)
        const int s = 32 * j + 16 * u + 4 * g;
        const f32x4 v = *reinterpret_cast<const f32x4*>(&lds_t[t * LD + s]);
        const f32x4 b = *reinterpret_cast<const f32x4*>(&lds_beta[s]);
        f32x4 w;
#pragma unroll
        for (int r = 0; r < 4; ++r) w[r] = s + r <= t ? v[r] * b[r] : 0.f;   // (above the diagonal nothing is written)
        *reinterpret_cast<f32x4*>(blob + C::kT + ((f * 2 + u) * 64 + lane) * 16) = w;
      }
    }
}

// A buffer at an address that is uniform over the workgroup.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer(const void* base, int bytes) {
  const uint64_t p = reinterpret_cast<uint64_t>(base);
  const uint32_t low = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)p);
  const uint32_t high = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(p >> 32));
  return __builtin_amdgcn_make_buffer_rsrc(reinterpret_cast<void*>((uint64_t)high << 32 | low), 0,
                                           __builtin_amdgcn_readfirstlane(bytes), 0x00020000);
}
__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t r, uint32_t offset) {
  return __builtin_amdgcn_raw_buffer_load_b128(r, (int)offset, 0, 0);
}

// The sequence that is the i-th longest, of up to 64: workgroups start in their order, and
// the long chains must not be the last (8192 tokens cut into eight prompts at random, 32
// heads of 128 x 128 bf16: 277 us by length, 309 as given).
__device__ __forceinline__ int longest(const Sequences& q, int i, int lane) {
  if (!q.offsets || q.seqs > 64 || q.seqs == 1) return i;
  int b, l = -1;
  if (lane < q.seqs) first_slot(q, lane, b, l);
  int rank = 0;
  for (int j = 0; j < q.seqs; ++j) {
    const int other = __builtin_amdgcn_readlane(l, j);
    rank += other > l || (other == l && j < lane) ? 1 : 0;
  }
  return (int)__builtin_ctzll(__builtin_amdgcn_ballot_w64(lane < q.seqs && rank == i));
}

// The pieces of a product's factor, 32 of its rows or columns: a lane's first four, then its second four
typedef u32x2 Halves[2][64];
__device__ __forceinline__ u32x4 both(const Halves& h, int lane) {
  const u32x2 lo = h[0][lane], hi = h[1][lane];
  return u32x4{lo[0], lo[1], hi[0], hi[1]};
}
template <int N>
__device__ __forceinline__ void put_four(Halves (&h)[N], int half, int lane, const f32x4& v) {
  uint32_t lo[N], hi[N];
  split(v[0], v[1], lo);
  split(v[2], v[3], hi);
#pragma unroll
  for (int q = 0; q < N; ++q) h[q][half][lane] = u32x2{lo[q], hi[q]};
}

// The chain of a sequence's chunks. Eight wavefronts share NC x 16 columns of one head's
// state. Four of them make U, the four others O and the state, of which each has a
// quarter of the rows in registers over the whole sequence; U and O each a tile of 16 of
// a chunk's tokens. A chunk is three steps, with a barrier after each; what a step needs
// of another wavefront passes through LDS:
//   1. K S0 and X = V - e^c K S0, from all pieces of S0 | O of the last chunk
//   2. U = T X, from all pieces of X                    | S0^T Q^T
//   3. the next chunk's K to LDS                        | S, from all pieces of U and all of K
// Everything else comes straight from memory into registers, a chunk ahead, each fetch
// where its wavefront waits for LDS anyway. K passes through LDS to be read as columns,
// in planes of four of each eight keys, so that such reads take whole runs of banks.
//
// Rows k of the state are spread over the lanes so that a lane's 8 of a step of 32
// follow one another, in the order in which a product takes 8 keys of a token: register
// r of lane group g in tile kt is row 32 (kt / 2) + 8 g + 4 (kt & 1) + r. Results of one
// product are then factors of the next as they are.
template <typename T, int DK, int PI, int PY, int NC>
__global__ __launch_bounds__(512) void delta_kernel(DeltaArgs a) {
  typedef Chunk<PY> C;
  constexpr int KS = DK / 32, KTW = DK / 64;   // steps of 32 keys, a wavefront's tiles of 16 rows
  constexpr int TS = kL / 32;
  constexpr int KEYS = 2 * PI * kL * DK * 2;
  constexpr int CH = NC == 1 ? 3 : 1;   // sums of a product that go side by side
  __shared__ __attribute__((aligned(16))) Halves lds_s[NC][KS][kPieces], lds_x[NC][TS][kPieces];
  __shared__ __attribute__((aligned(16))) Halves lds_w[NC][TS][kPieces], lds_u[NC][TS][PY];
  __shared__ __attribute__((aligned(16))) uint8_t lds_k[2][PI][KS][2][kL * 32];
  __shared__ __attribute__((aligned(16))) u32x2 lds_v[PI == 1 ? 4 : 1][NC][64];
  __shared__ int lds_first[2][NC * 16];   // first token of a column whose X is not finite
  __shared__ int lds_any[2];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6) & 3;
  const bool makes_u = __builtin_amdgcn_readfirstlane(tid >> 8) == 0;
  const int n16 = lane & 15, g = lane >> 4;
  // Workgroups go round the 8 XCDs: those of one head and sequence, which read the
  // same chunks, go to one XCD's cache.
  const int id = blockIdx.x >> 3;
  const int unit = id / a.vblocks * 8 + (blockIdx.x & 7);
  if (unit >= a.units) return;
  const int v0 = (id % a.vblocks) * 16 * NC;
  const int h = unit % a.l.H, hk = h / a.l.per_key;
  const int sq = __builtin_amdgcn_readfirstlane(longest(a.l.s, unit / a.l.H, lane));
  const int dk = a.l.dk, dv = a.l.dv;
  int begin, len;
  const int slot0 = __builtin_amdgcn_readfirstlane(first_slot(a.l.s, sq, begin, len));
  begin = __builtin_amdgcn_readfirstlane(begin), len = __builtin_amdgcn_readfirstlane(len);
  const int chunks = (len + kL - 1) / kL;
  if (chunks == 0 && a.l.state_in) return;
  if (chunks == 1 && len <= kFew) return;   // (the first kernel has it)

  const int t16 = 16 * wave;   // its tokens
  auto rows_of = [&](int c) { return max(min(len - c * kL, kL), 0); };   // (none past the last chunk)
  const size_t blob_step = (size_t)a.l.H * C::kBytes;
  const uint8_t* blob = a.chunks + ((size_t)slot0 * a.l.H + h) * C::kBytes;
  auto blob_of = [&](int c) { return buffer(blob, c < chunks ? C::kBytes : 0); };
  // keys or queries: rows as they are, or the pieces that the first kernel left
  const int row_bytes = PI == 1 ? (int)((makes_u ? a.l.k_stride : a.l.q_stride) * sizeof(T)) : DK * 2;
  const uint8_t* key_at = PI == 1 ? reinterpret_cast<const uint8_t*>(makes_u ? a.l.k : a.l.q) + (int64_t)begin * row_bytes + (size_t)hk * dk * 2
                                  : a.keys + ((size_t)slot0 * (a.l.H / a.l.per_key) + hk) * KEYS + (makes_u ? 0 : KEYS / 2);
  const size_t key_step = PI == 1 ? (size_t)kL * row_bytes : (size_t)(a.l.H / a.l.per_key) * KEYS;
  uint32_t key_off[KS];
#pragma unroll
  for (int i = 0; i < KS; ++i)
    key_off[i] = 32 * i + 8 * g < dk ? (uint32_t)((t16 + n16) * row_bytes + 64 * i + 16 * g) : kOutside;
  u32x4 kf[KS][PI];   // of token n16, eight keys or queries
  auto fetch_keys = [&](int c) {
    const auto r = buffer(key_at, PI == 1 ? rows_of(c) * row_bytes : c < chunks ? KEYS / 2 : 0);
    key_at += key_step;
#pragma unroll
    for (int i = 0; i < KS; ++i)
#pragma unroll
      for (int p = 0; p < PI; ++p) kf[i][p] = load16(r, key_off[i] + p * kL * DK * 2);
  };
  if (tid < 2 * NC * 16) lds_first[tid / (NC * 16)][tid % (NC * 16)] = kL;
  if (tid < 2) lds_any[tid] = 0;
  // a lane's place as it names the run of four that it reads columns of: tokens 4 g .. 4 g + 3
  const int run = (4 * g + (n16 >> 2)) * 32 + (n16 & 3) * 8;

  if (makes_u) {
    // ---------------------------------------------------------------- U
    const uint8_t* v_at = reinterpret_cast<const uint8_t*>(a.l.v) + ((int64_t)begin * a.l.v_stride + (size_t)h * dv) * sizeof(T);
    const int vrow = (int)(a.l.v_stride * sizeof(T));
    // v of tokens 4 g + r, this lane's column: bf16 rows are read whole, four columns a lane, and pass through LDS
    uint32_t voff[NC][PI == 1 ? 1 : 4];
    u32x2 vrows[NC];
    uint32_t vn[NC][4];
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      if constexpr (PI == 1) {
        const int col = v0 + 16 * n + 4 * (lane & 3);
        voff[n][0] = col < dv ? (uint32_t)((t16 + (lane >> 2)) * vrow + col * 2) : kOutside;
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          voff[n][r] = v0 + 16 * n + n16 < dv ? (uint32_t)((t16 + 4 * g + r) * vrow + (v0 + 16 * n + n16) * 4) : kOutside;
      }
    }
    auto fetch_v = [&](int c) {
      const auto rV = buffer(v_at, rows_of(c) * vrow);
      v_at += (size_t)kL * vrow;
#pragma unroll
      for (int n = 0; n < NC; ++n) {
        if constexpr (PI == 1) {
          vrows[n] = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(rV, (int)voff[n][0], 0, 0));
        } else {
#pragma unroll
          for (int r = 0; r < 4; ++r) vn[n][r] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(rV, (int)voff[n][r], 0, 0);
        }
      }
    };
    // its tile's fragments of T, zeros for tokens s behind them; the next chunk's as loaded
    u32x4 tf[TS][kPieces], tn[TS][2];
    f32x4 to, from;          // decays to tokens 4 g + r, and from them to the chunk's end
    auto fetch_t = [&](int c) {
      const auto r = blob_of(c);
#pragma unroll
      for (int j = 0; j < TS; ++j)
#pragma unroll
        for (int u = 0; u < 2; ++u)
          tn[j][u] = load16(r, 2 * j + u <= wave ? (uint32_t)(C::kT + (C::fragment(wave, j) * 2 + u) * 1024 + lane * 16) : kOutside);
    };
    auto fetch_decays = [&](int c) {
      const auto r = blob_of(c);
      to = __builtin_bit_cast(f32x4, load16(r, C::kTo + 4 * t16 + 16 * g));
      from = __builtin_bit_cast(f32x4, load16(r, C::kFrom + 4 * t16 + 16 * g));
    };
    auto split_t = [&]() {
#pragma unroll
      for (int j = 0; j < TS; ++j)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const f32x4 v = __builtin_bit_cast(f32x4, tn[j][u]);
          uint32_t lo[kPieces], hi[kPieces];
          split(v[0], v[1], lo);
          split(v[2], v[3], hi);
#pragma unroll
          for (int q = 0; q < kPieces; ++q) tf[j][q][2 * u] = lo[q], tf[j][q][2 * u + 1] = hi[q];
        }
    };
    // K's planes, and v's columns
    auto put_keys = [&](int c) {
      uint8_t* const put = &lds_k[c & 1][0][0][0][(t16 + n16) * 32 + g * 8];
#pragma unroll
      for (int i = 0; i < KS; ++i)
#pragma unroll
        for (int p = 0; p < PI; ++p) {
          uint8_t* const at = put + (p * KS + i) * 2 * kL * 32;
          *reinterpret_cast<u32x2*>(at) = u32x2{kf[i][p][0], kf[i][p][1]};
          *reinterpret_cast<u32x2*>(at + kL * 32) = u32x2{kf[i][p][2], kf[i][p][3]};
        }
      if constexpr (PI == 1) {
#pragma unroll
        for (int n = 0; n < NC; ++n) lds_v[wave][n][lane] = vrows[n];
#pragma unroll
        for (int n = 0; n < NC; ++n) {
          const u32x2 w = read_tr(reinterpret_cast<const uint8_t*>(lds_v[wave][n]) + run);
          vn[n][0] = w[0] << 16, vn[n][1] = w[0] & 0xFFFF0000u, vn[n][2] = w[1] << 16, vn[n][3] = w[1] & 0xFFFF0000u;
        }
      }
    };

    fetch_t(0);
    fetch_decays(0);
    fetch_keys(0);
    fetch_v(0);
    split_t();
    blob += blob_step;
    fetch_t(1);
    put_keys(0);
    __syncthreads();
    for (int c = 0; c < chunks; ++c) {
      const int par = c & 1;
      // ---- 1: K S0 (rows t, columns v), X = V - e^c K S0
      f32x4 x[NC][CH];
#pragma unroll
      for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int i = 0; i < CH; ++i) x[n][i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        u32x4 sf[NC][kPieces];
#pragma unroll
        for (int n = 0; n < NC; ++n)
#pragma unroll
          for (int q = 0; q < kPieces; ++q) sf[n][q] = both(lds_s[n][i][q], lane);
        // (products that follow one another go to different sums: one waits for the last to its own)
#pragma unroll
        for (int p = 0; p < PI; ++p)
#pragma unroll
          for (int q = 0; q < kPieces; ++q)
#pragma unroll
            for (int n = 0; n < NC; ++n)
              if (p + q < 3) x[n][(p + 2 * q) % CH] = mfma(kf[i][p], sf[n][q], x[n][(p + 2 * q) % CH]);
      }
      float odd = 0.f;   // 0 X, a NaN where X is not finite
#pragma unroll
      for (int n = 0; n < NC; ++n) {
#pragma unroll
        for (int i = 1; i < CH; ++i) x[n][0] += x[n][i];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          x[n][0][r] = __builtin_fmaf(-to[r], x[n][0][r], __uint_as_float(vn[n][r]));
          odd = __builtin_fmaf(0.f, x[n][0][r], odd);
        }
      }
      // A product takes all tokens, with weights of zero for later ones: an X that is not
      // finite is taken out, and its column NaN from its token on
      if (__builtin_amdgcn_ballot_w64(odd != odd)) {
#pragma unroll
        for (int n = 0; n < NC; ++n)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if ((__float_as_uint(x[n][0][r]) & 0x7F800000u) == 0x7F800000u) {
              x[n][0][r] = 0.f;
              atomicMin(&lds_first[par][16 * n + n16], t16 + 4 * g + r);
            }
        lds_any[par] = 1;
      }
#pragma unroll
      for (int n = 0; n < NC; ++n) put_four(lds_x[n][wave >> 1], wave & 1, lane, x[n][0]);
      __syncthreads();
      // ---- 2: U = T X
      f32x4 u[NC][CH];
#pragma unroll
      for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int i = 0; i < CH; ++i) u[n][i] = f32x4{0.f, 0.f, 0.f, 0.f};
      u32x4 xf[NC][TS][kPieces];
#pragma unroll
      for (int j = 0; j < TS; ++j)
#pragma unroll
        for (int n = 0; n < NC; ++n)
#pragma unroll
          for (int q = 0; q < kPieces; ++q) xf[n][j][q] = both(lds_x[n][j][q], lane);
      __builtin_amdgcn_sched_barrier(0);
      fetch_keys(c + 1);
      fetch_v(c + 1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < TS; ++j)
#pragma unroll
        for (int p = 0; p < kPieces; ++p)
#pragma unroll
          for (int q = 0; q < kPieces; ++q)
#pragma unroll
            for (int n = 0; n < NC; ++n)
              if (p + q < 3) u[n][(p + 2 * q) % CH] = mfma(tf[j][p], xf[n][j][q], u[n][(p + 2 * q) % CH]);
#pragma unroll
      for (int n = 0; n < NC; ++n) {
#pragma unroll
        for (int i = 1; i < CH; ++i) u[n][0] += u[n][i];
        put_four(lds_w[n][wave >> 1], wave & 1, lane, u[n][0] * from);
        put_four(lds_u[n][wave >> 1], wave & 1, lane, u[n][0]);
      }
      __syncthreads();
      // ---- 3
      if (tid < NC * 16) lds_first[par ^ 1][tid] = kL;
      if (tid == NC * 16) lds_any[par ^ 1] = 0;
      fetch_decays(c + 1);
      split_t();
      blob += blob_step;
      fetch_t(c + 2);
      put_keys(c + 1);
      __syncthreads();
    }
    return;
  }
  // ---------------------------------------------------------------- O and the state
  float* const st = a.l.state + ((size_t)sq * a.l.H + h) * dk * dv + v0 + n16;
  auto state_row = [&](int kt, int r) {
    const int t = wave * KTW + kt;
    return 32 * (t >> 1) + 8 * g + 4 * (t & 1) + r;
  };
  f32x4 S[NC][KTW];
#pragma unroll
  for (int n = 0; n < NC; ++n)
#pragma unroll
    for (int kt = 0; kt < KTW; ++kt) {
      S[n][kt] = f32x4{0.f, 0.f, 0.f, 0.f};
      if (a.l.state_in) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (state_row(kt, r) < dk && v0 + 16 * n + n16 < dv) S[n][kt][r] = st[(size_t)state_row(kt, r) * dv + 16 * n];
      }
    }
  auto put_state = [&]() {
#pragma unroll
    for (int n = 0; n < NC; ++n)
#pragma unroll
      for (int kt = 0; kt < KTW; ++kt) put_four(lds_s[n][(wave * KTW + kt) >> 1], (wave * KTW + kt) & 1, lane, S[n][kt]);
  };
  uint8_t* o_at = reinterpret_cast<uint8_t*>(a.l.o) + ((int64_t)begin * a.l.o_stride + (size_t)h * dv) * sizeof(T);
  const int orow = (int)(a.l.o_stride * sizeof(T));
  uint32_t ooff[NC];
#pragma unroll
  for (int n = 0; n < NC; ++n)
    ooff[n] = v0 + 16 * n + 4 * g < dv ? (uint32_t)((t16 + n16) * orow + (v0 + 16 * n + 4 * g) * (int)sizeof(T)) : kOutside;
  u32x4 pf[TS][PY];   // its tile's fragments of P^T, zeros for tokens s behind them
  float to = 0.f;     // decay to token n16
  float decay = 0.f;  // e^{c_n}
  int bad = kL;       // the chunk's first token whose key or gates are not finite
  auto fetch_p = [&](int c) {
    const auto r = blob_of(c);
#pragma unroll
    for (int j = 0; j < TS; ++j)
#pragma unroll
      for (int p = 0; p < PY; ++p)
        pf[j][p] = load16(r, 2 * j <= wave ? (uint32_t)(C::kP + (C::fragment(wave, j) * PY + p) * 1024 + lane * 16) : kOutside);
    to = __uint_as_float((uint32_t)__builtin_amdgcn_raw_buffer_load_b32(r, C::kTo + 4 * t16 + 4 * n16, 0, 0));
    decay = __uint_as_float((uint32_t)__builtin_amdgcn_raw_buffer_load_b32(r, C::kDecay, 0, 0));
    bad = __builtin_amdgcn_raw_buffer_load_b32(r, C::kBad, 0, 0);
  };
  f32x4 o[NC];   // S0^T Q^T
  // O^T = e^c S0^T Q^T + U^T P^T of a chunk (before the first there are no rows)
  auto finish = [&](int c) {
    const int par = c & 1;
    const int flag = lds_any[par];
    u32x4 uf[NC][TS][PY];
#pragma unroll
    for (int n = 0; n < NC; ++n)
#pragma unroll
      for (int j = 0; j < TS; ++j)
#pragma unroll
        for (int q = 0; q < PY; ++q) uf[n][j][q] = both(lds_u[n][j][q], lane);
    f32x4 y[NC][CH];
#pragma unroll
    for (int n = 0; n < NC; ++n)
#pragma unroll
      for (int i = 0; i < CH; ++i) y[n][i] = i == 0 ? o[n] * to : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < TS; ++j)
#pragma unroll
      for (int p = 0; p < PY; ++p)
#pragma unroll
        for (int q = 0; q < PY; ++q)
#pragma unroll
          for (int n = 0; n < NC; ++n)
            // (of two pieces each all four: without the last 2^-16 more of a term could be missing)
            if (p + q < 3) y[n][(p + 2 * q) % CH] = mfma(uf[n][j][q], pf[j][p], y[n][(p + 2 * q) % CH]);
    settle();
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      o[n] = y[n][0];
#pragma unroll
      for (int i = 1; i < CH; ++i) o[n] += y[n][i];
    }
    if (__builtin_amdgcn_readfirstlane(flag | (bad < kL)) != 0)
#pragma unroll
      for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (t16 + n16 >= min(bad, lds_first[par][16 * n + 4 * g + r])) o[n][r] = __builtin_nanf("");
    const auto rO = buffer(o_at, c < 0 ? 0 : rows_of(c) * orow);
    if (c >= 0) o_at += (size_t)kL * orow;
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      if constexpr (PI == 1)
        __builtin_amdgcn_raw_buffer_store_b64(u32x2{bf16_pair(o[n][0], o[n][1]), bf16_pair(o[n][2], o[n][3])}, rO, (int)ooff[n], 0, 0);
      else
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, o[n]), rO, (int)ooff[n], 0, 0);
    }
  };
#pragma unroll
  for (int j = 0; j < TS; ++j)
#pragma unroll
    for (int p = 0; p < PY; ++p) pf[j][p] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
  for (int n = 0; n < NC; ++n) o[n] = f32x4{0.f, 0.f, 0.f, 0.f};
  fetch_keys(0);
  put_state();
  __syncthreads();
  for (int c = 0; c < chunks; ++c) {
    const int par = c & 1;
    // ---- 1: O of the last chunk
    finish(c - 1);
    fetch_p(c);
    blob += blob_step;
    __syncthreads();
    // ---- 2: S0^T Q^T (rows v, columns t)
    f32x4 y[NC][CH];
#pragma unroll
    for (int n = 0; n < NC; ++n)
#pragma unroll
      for (int i = 0; i < CH; ++i) y[n][i] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      u32x4 sf[NC][PY];
#pragma unroll
      for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int q = 0; q < PY; ++q) sf[n][q] = both(lds_s[n][i][q], lane);
#pragma unroll
      for (int p = 0; p < PI; ++p)
#pragma unroll
        for (int q = 0; q < PY; ++q)
#pragma unroll
          for (int n = 0; n < NC; ++n)
            if (p + q < 3) y[n][(i + p + 2 * q) % CH] = mfma(sf[n][q], kf[i][p], y[n][(i + p + 2 * q) % CH]);
    }
    settle();
#pragma unroll
    for (int n = 0; n < NC; ++n) {
      o[n] = y[n][0];
#pragma unroll
      for (int i = 1; i < CH; ++i) o[n] += y[n][i];
    }
    __syncthreads();
    // ---- 3: S <- e^{c_n} S0 + K^T (e^{c_n - c} U)
    const int flag = lds_any[par];
    const uint8_t* const k_get = &lds_k[par][0][0][0][run];
    f32x4 add[NC][KTW];
#pragma unroll
    for (int n = 0; n < NC; ++n)
#pragma unroll
      for (int kt = 0; kt < KTW; ++kt) add[n][kt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < TS; ++j) {
      u32x4 wf[NC][kPieces];
#pragma unroll
      for (int n = 0; n < NC; ++n)
#pragma unroll
        for (int q = 0; q < kPieces; ++q) wf[n][q] = both(lds_w[n][j][q], lane);
#pragma unroll
      for (int p = 0; p < PI; ++p) {
        u32x4 kc[KTW];
#pragma unroll
        for (int kt = 0; kt < KTW; ++kt) {
          const int t = wave * KTW + kt;
          const uint8_t* const at = k_get + ((p * KS + (t >> 1)) * 2 + (t & 1)) * kL * 32 + 32 * j * 32;
          const u32x2 lo = read_tr(at), hi = read_tr(at + 16 * 32);
          kc[kt] = u32x4{lo[0], lo[1], hi[0], hi[1]};
        }
#pragma unroll
        for (int q = 0; q < kPieces; ++q)
#pragma unroll
          for (int kt = 0; kt < KTW; ++kt)
#pragma unroll
            for (int n = 0; n < NC; ++n)
              if (p + q < 3) add[n][kt] = mfma(kc[kt], wf[n][q], add[n][kt]);
      }
      if (j == 0) fetch_keys(c + 1);
    }
#pragma unroll
    for (int n = 0; n < NC; ++n)
#pragma unroll
      for (int kt = 0; kt < KTW; ++kt)
#pragma unroll
        for (int r = 0; r < 4; ++r) S[n][kt][r] = __builtin_fmaf(S[n][kt][r], decay, add[n][kt][r]);
    if (__builtin_amdgcn_readfirstlane(flag | (bad < kL)) != 0)
#pragma unroll
      for (int n = 0; n < NC; ++n)
        if (min(bad, lds_first[par][16 * n + n16]) < kL)
#pragma unroll
          for (int kt = 0; kt < KTW; ++kt)
#pragma unroll
            for (int r = 0; r < 4; ++r) S[n][kt][r] = __builtin_nanf("");
    put_state();
    __syncthreads();
  }
  if (chunks > 0) finish(chunks - 1);
#pragma unroll
  for (int n = 0; n < NC; ++n)
#pragma unroll
    for (int kt = 0; kt < KTW; ++kt)
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (state_row(kt, r) < dk && v0 + 16 * n + n16 < dv) st[(size_t)state_row(kt, r) * dv + 16 * n] = S[n][kt][r];
}

typedef void (*DeltaFn)(DeltaArgs);

struct DeltaPlan {
  DeltaFn prepare, scan;
  int64_t slots, units, vblocks;
  bool few;   // no sequence is longer than kFew
  size_t chunk_bytes, bytes;
};

// Column tiles of a workgroup. More of them share a chunk's reading, fewer leave a shorter
// chain. A chunk takes a workgroup of one, two and four tiles 1.7, 2.55 and 4.4 us, and a
// compute unit that has others to go on with 1.65, 1.33 and 1.26 us a tile (128 x 128
// bf16): the longest sequence takes its chunks one after another, and all that the
// 256 compute units share. By the longer of the two, us, the first tiles chosen: 8192 tokens
// of 32 heads one 301, two 382, four 613; of 64 heads two 477, one 555, four 662; of 128 four
// 838, two 876, one 1041. The same times decide for the other types and widths: of bf16 with d_k
// 64, 128 and 256 and fp32 with 64 and 128, 4096 tokens of 16 to 128 heads, 8 and 16 prompts of 512
// and 64 of 256, the tiles chosen were the fastest of all in each case, or within 2% of it (4096
// tokens of 32 heads of 128 x 128 fp32 one 354, two 398; of 64 two 497, one 688; of 256 x 128 bf16
// one 220, two 308, and two 347, one 430; of 64 x 64 bf16, 128 heads, two 226, one 278, four 315).
template <typename T, int DK, int PI, int PY>
void pick_delta(DeltaPlan& w, const rsq_linear_attn* p) {
  w.prepare = delta_prepare_kernel<T, DK, PI, PY>;
  w.units = (int64_t)p->seqs * p->heads;
  const int64_t tiles = ceil_div(p->d_v, 16);
  // a sequence of len rows has ceil(len / kL) chunks; with their rows apart, at most tokens / kL + seqs in all
  w.slots = p->tokens / kL + p->seqs;
  constexpr int kMost = PI > 1 || DK > 128 ? 2 : 4;   // (four take more LDS or registers than there are)
  constexpr float kChain[3] = {1.7f, 2.55f, 4.4f}, kTile[3] = {1.65f, 1.33f, 1.26f};
  float best = 0.f;
  int nc = 0;
  for (int i = 0; 1 << i <= kMost; ++i) {
    const float shared = ((float)p->tokens / kL + .5f * p->seqs) * (float)p->heads * (float)(ceil_div(tiles, 1 << i) << i) * kTile[i] / 256.f;
    const float chain = (float)ceil_div(p->max_len, kL) * kChain[i], time = chain > shared ? chain : shared;
    if (nc == 0 || time < best) best = time, nc = 1 << i;
  }
  w.scan = nc == 1 ? delta_kernel<T, DK, PI, PY, 1> : nc == 2 ? delta_kernel<T, DK, PI, PY, 2> : delta_kernel<T, DK, PI, PY, kMost>;
  w.vblocks = ceil_div(tiles, nc);
  w.chunk_bytes = (size_t)w.slots * p->heads * Chunk<PY>::kBytes;
  w.few = p->max_len <= kFew;
  w.bytes = w.few ? 0 : w.chunk_bytes + (PI > 1 ? (size_t)w.slots * p->key_heads * 2 * PI * kL * DK * 2 : 0);
}

rsq_status plan_delta(const rsq_linear_attn* p, DeltaPlan& w) {
  if (p->dtype == RSQ_BF16) {
    if (p->d_k <= 64) pick_delta<Bf16, 64, 1, 2>(w, p);
    else if (p->d_k <= 128) pick_delta<Bf16, 128, 1, 2>(w, p);
    else pick_delta<Bf16, 256, 1, 2>(w, p);
  } else {
    if (p->d_k <= 64) pick_delta<float, 64, 3, 3>(w, p);
    else pick_delta<float, 128, 3, 3>(w, p);
  }
  if (const rsq_status s = check_blocks(w.slots * p->heads, 256)) return s;
  return check_blocks(ceil_div(w.units, 8) * 8 * w.vblocks, 512);
}

}  // namespace

rsq_status delta_workspace(const rsq_linear_attn* p, size_t* bytes) {
  DeltaPlan w;
  if (const rsq_status s = plan_delta(p, w)) return s;
  *bytes = w.bytes;
  return RSQ_OK;
}

rsq_status run_delta(const rsq_linear_attn* p, const LinearArgs& l, void* stream) {
  DeltaPlan w;
  if (const rsq_status s = plan_delta(p, w)) return s;
  if (w.bytes > 0) {
    if (!p->workspace || !aligned(p->workspace, 16)) return fail(RSQ_E_INVALID, "workspace is NULL or not 16-byte aligned");
    if (p->workspace_bytes < w.bytes)
      return fail(RSQ_E_BUFFER, "workspace has %zu bytes, the call needs %zu", p->workspace_bytes, w.bytes);
  }
  DeltaArgs a{};
  a.l = l;
  a.chunks = static_cast<uint8_t*>(p->workspace);
  a.keys = a.chunks + w.chunk_bytes;
  a.vblocks = (int32_t)w.vblocks, a.units = (int32_t)w.units;
  if (p->max_len > 0) {
    // Columns side by side where all sequences are short or there are few of them (a chunk takes the first only).
    // One of 64 tokens and, of eight each, one (of 16 heads, 48 workgroups) 17 us so, 24 otherwise; four (of 32
    // heads, 192) 28.5, 33; eight (352) 31, 36; 16 (640) 38, 42; but 32 (1216) 64.6, 62.
    const int64_t across = w.few || w.slots * p->heads <= 512 ? ceil_div(p->d_v, 64) : 1;
    hipLaunchKernelGGL(w.prepare, dim3((unsigned)(w.slots * p->heads), (unsigned)across), dim3(256), 0, (hipStream_t)stream, a);
    if (const rsq_status s = launched("delta rule, chunks")) return s;
    if (w.few && (p->state_in || !p->offsets)) return RSQ_OK;   // (no chain, and no empty sequence's state to clear)
  }
  const int64_t blocks = ceil_div(w.units, 8) * 8 * w.vblocks;
  hipLaunchKernelGGL(w.scan, dim3((unsigned)blocks), dim3(512), 0, (hipStream_t)stream, a);
  return launched("delta rule");
}

}  // namespace rsq

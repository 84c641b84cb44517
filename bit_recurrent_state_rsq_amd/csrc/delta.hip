// Attention with the delta rule over prompts (linear.hpp has the recurrence), in
// chunks of L tokens. With c_t the sum of log a over a chunk's tokens up to t, S0
// the state before the chunk and n its last token, the chunk's u solve
//   u_t + sum_{s < t} A_ts u_s = b_t (v_t - e^{c_t} S0^T k_t),  A_ts = b_t e^{c_t - c_s} (k_t . k_s),
// so that with T = (1 + A)^-1 diag(b), which does not depend on the state,
//   X = V - e^c K S0,   U = T X,
//   O = e^c Q S0 + P U,   P_ts = e^{c_t - c_s} (q_t . k_s) for s <= t,
//   S <- e^{c_n} S0 + K^T (e^{c_n - c} U).
// delta_prepare_kernel makes T and P of all chunks side by side; delta_kernel then
// follows the state through a sequence's chunks.
#include <algorithm>

#include "chunk.hpp"
#include "host_util.hpp"
#include "linear.hpp"

namespace rsq {
namespace {

constexpr int kPieces = 3;   // of fp32 factors that reach the state

struct DeltaArgs {
  LinearArgs l;
  uint8_t* chunks;    // [slot][head] what a chunk's tokens give (Chunk)
  uint8_t* keys;      // fp32: [slot][key head][K, Q][pieces] tiles as LDS has them
  int32_t slots;      // chunks of all sequences, at most
  int32_t vblocks;    // column blocks of a head
  int32_t units;      // sequences x heads
};

// What the first kernel leaves of a chunk and head for the second: fragments of T
// (pieces of its fp32) and P^T as products of 32 tokens s take them, those with an
// s <= t only, and the decays.
template <int L, int PY>
struct Chunk {
  static constexpr int kTiles = L / 16;                  // of tokens t
  static constexpr int kFragments = L == 64 ? 6 : 2;
  // fragment of tokens t in tile e, s in the j-th 32
  static __device__ constexpr int fragment(int e, int j) { return e < 2 ? e : 2 * e - 2 + j; }
  static constexpr int kT = 0, kP = kFragments * kPieces * 1024, kGates = kP + kFragments * PY * 1024;
  static constexpr int kBytes = kGates + 1024;
  // floats of the gates: e^{c_t}, e^{c_n - c_t}; then e^{c_n}; the first token whose key or gate is not finite
  static constexpr int kTo = 0, kFrom = 64, kDecay = 128, kBad = 129;
};

// Chunk j of a sequence that begins at row b is slot b / L + s + j: those of the
// sequences before it end below that, whatever their lengths.
template <int L>
__device__ __forceinline__ int first_slot(const Sequences& q, int s, int& begin, int& len) {
  int64_t n;
  begin = (int)seq_range(q, s, n);
  len = (int)n;
  return begin / L + s;
}

// The sequence of a slot: the last one whose first slot is not above it. 64 sequences
// are looked at at a time, a 64th of those left apart.
template <int L>
__device__ __forceinline__ bool find_chunk(const Sequences& q, int slot, int lane, int& begin, int& len, int& chunk) {
  int lo = 0, n = q.seqs;
  for (;;) {
    const int step = (n + 63) / 64, s = lo + lane * step;
    int b = 0, l = 0;
    const bool below = lane * step < n && first_slot<L>(q, s, b, l) <= slot;
    const uint64_t hit = __builtin_amdgcn_ballot_w64(below);
    if (!hit) return false;
    const int last = 63 - __builtin_clzll(hit);
    if (step == 1) {
      begin = __builtin_amdgcn_readlane(b, last), len = __builtin_amdgcn_readlane(l, last);
      chunk = slot - (begin / L + lo + last);
      return chunk * L < len;
    }
    n = min(step, n - last * step);
    lo += last * step;
  }
}

__device__ __forceinline__ float exp2_of(double c) { return __builtin_amdgcn_exp2f((float)c); }

// One chunk of one head. K K^T and Q K^T on the matrix cores (exact products of the
// inputs' pieces); the inverse in fp32: 16 x 16 blocks on the diagonal by
// substitution, a column a lane, then the blocks below them, diagonal by diagonal,
// T_ij = -T_ii sum_k A_ik T_kj, by fp32 products.
template <typename T, int DK, int L, int PI, int PY>
__global__ __launch_bounds__(256) void delta_prepare_kernel(DeltaArgs a) {
  typedef Tile<DK> TB;
  typedef Chunk<L, PY> C;
  constexpr int TT = C::kTiles, KS = DK / 32, LD = L + 4;
  constexpr int BB = L * TB::kBytes;
  constexpr int KEYS = 2 * PI * BB, INV = L * LD * 4;
  // K and Q, and once their products are there, the inverse
  __shared__ __attribute__((aligned(16))) uint8_t raw[KEYS > INV ? KEYS : INV];
  __shared__ __attribute__((aligned(16))) float lds_a[L * LD];
  __shared__ double lds_c[L];
  __shared__ __attribute__((aligned(16))) float lds_beta[L];
  __shared__ int lds_bad;
  uint8_t* const lds_k = raw;
  uint8_t* const lds_q = raw + PI * BB;
  float* const lds_t = reinterpret_cast<float*>(raw);

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n16 = lane & 15, g = lane >> 4;
  const int h = blockIdx.x % a.l.H;
  const int slot = blockIdx.x / a.l.H;
  int begin, len, chunk;
  if (!find_chunk<L>(a.l.s, slot, lane, begin, len, chunk)) return;
  begin = __builtin_amdgcn_readfirstlane(begin), len = __builtin_amdgcn_readfirstlane(len);
  const int t0 = __builtin_amdgcn_readfirstlane(chunk) * L;
  const int hk = h / a.l.per_key, dk = a.l.dk;
  uint8_t* const blob = a.chunks + ((size_t)slot * a.l.H + h) * C::kBytes;

  // ---- rows to LDS
  constexpr int NB = L * (DK / 8) / 256, RB = 256 / (DK / 8);
  const int row0 = tid / (DK / 8), piece = tid % (DK / 8);
  const int krow = (int)(a.l.k_stride * sizeof(T)), qrow = (int)(a.l.q_stride * sizeof(T));
  Vec8<T, PI> rk[NB], rq[NB];
  {
    const ChunkRows<L> rK(reinterpret_cast<const T*>(a.l.k) + begin * a.l.k_stride + (size_t)hk * dk, krow, t0, len);
    const ChunkRows<L> rQ(reinterpret_cast<const T*>(a.l.q) + begin * a.l.q_stride + (size_t)hk * dk, qrow, t0, len);
    const bool in = piece * 8 < dk;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      rk[i].load(rK, in ? (uint32_t)((row0 + i * RB) * krow + piece * 8 * (int)sizeof(T)) : kOutside);
      rq[i].load(rQ, in ? (uint32_t)((row0 + i * RB) * qrow + piece * 8 * (int)sizeof(T)) : kOutside);
    }
  }
  const bool valid = lane < L && t0 + lane < len;
  float al = 1.f, be = 0.f;
  if (wave == 0 && valid) {
    const int64_t row = (int64_t)begin + t0 + lane;
    if (a.l.alpha) al = a.l.alpha[row * a.l.alpha_stride + h];
    be = a.l.beta[row * a.l.beta_stride + h];
  }
  if (tid == 0) lds_bad = L;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    const int row = row0 + i * RB;
    const uint32_t at = TB::at(row, piece);
    u32x4 pk[PI], pq[PI];
    rk[i].pieces(pk);
    rq[i].pieces(pq);
#pragma unroll
    for (int p = 0; p < PI; ++p) {
      *reinterpret_cast<u32x4*>(lds_k + p * BB + at) = pk[p];
      *reinterpret_cast<u32x4*>(lds_q + p * BB + at) = pq[p];
    }
    if (rk[i].bad_bits() & (PI == 1 ? 0x80008000u : 0x80000000u)) atomicMin(&lds_bad, row);
    if constexpr (PI > 1) {
      if (h % a.l.per_key == 0) {
        uint8_t* const to = a.keys + ((size_t)slot * (a.l.H / a.l.per_key) + hk) * KEYS + at;
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
    const int bad = min(lds_bad, odd ? (int)__builtin_ctzll(odd) : L);
    const bool in = valid && lane < bad;
    double cum = in ? log2((double)al) : 0.;
    cum = cum < -2000. ? -2000. : cum;   // (as good as nothing of an fp32 state is left)
    cum = wave_scan(cum);
    const double last = lane63(cum);
    float* const gates = reinterpret_cast<float*>(blob + C::kGates);
    if (lane < L) {
      lds_c[lane] = cum;
      lds_beta[lane] = in ? be : 0.f;
      gates[C::kTo + lane] = exp2_of(cum);
      gates[C::kFrom + lane] = exp2_of(last - cum);
    }
    if (lane == 0) {
      gates[C::kDecay] = exp2_of(last);
      reinterpret_cast<int*>(gates)[C::kBad] = bad;
      lds_bad = bad;
    }
  }
  __syncthreads();
  const int bad = lds_bad;
  // ---- rows s, columns t, of the products with K (for A) and with Q (P^T): two tiles
  // of s at a time, a step of the products that take P
  const uint32_t a_frag = TB::fragment(lane);
  auto products = [&](int e, bool keys) {
    const uint8_t* const cols = keys ? lds_k : lds_q;
    const int t = 16 * e + n16;
    const double ct = lds_c[t];
    const float bt = lds_beta[t];
    u32x4 cf[KS][PI];
#pragma unroll
    for (int i = 0; i < KS; ++i)
#pragma unroll
      for (int p = 0; p < PI; ++p) cf[i][p] = *reinterpret_cast<const u32x4*>(cols + p * BB + 16 * e * TB::kBytes + (a_frag ^ (i << 6)));
#pragma unroll
    for (int j = 0; j < L / 32; ++j) {
      if (2 * j > e) continue;
      f32x4 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int i = 0; i < KS; ++i)
#pragma unroll
        for (int p = 0; p < PI; ++p)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const u32x4 kf = *reinterpret_cast<const u32x4*>(lds_k + p * BB + (32 * j + 16 * u) * TB::kBytes + (a_frag ^ (i << 6)));
#pragma unroll
            for (int q = 0; q < PI; ++q)
              if (p + q < 3) acc[u] = mfma(kf, cf[i][q], acc[u]);
          }
      settle();
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int s = 32 * j + 16 * u + 4 * g + r;
          // later tokens, and those from a bad one on, have no part whatever their products are
          const bool in = s < bad && (keys ? s < t && t < bad : s <= t);
          const float d = in ? exp2_of(ct - lds_c[s]) : 0.f;
          acc[u][r] = in ? acc[u][r] * d : 0.f;
          if (keys) acc[u][r] *= bt;
        }
      if (keys) {
#pragma unroll
        for (int u = 0; u < 2; ++u) *reinterpret_cast<f32x4*>(&lds_a[t * LD + 32 * j + 16 * u + 4 * g]) = acc[u];
      } else {
        u32x4 pf[PY];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          uint32_t lo[PY], hi[PY];
          split_pair<PY>(acc[u][0], acc[u][1], lo);
          split_pair<PY>(acc[u][2], acc[u][3], hi);
#pragma unroll
          for (int q = 0; q < PY; ++q) pf[q][2 * u] = lo[q], pf[q][2 * u + 1] = hi[q];
        }
#pragma unroll
        for (int q = 0; q < PY; ++q)
          *reinterpret_cast<u32x4*>(blob + C::kP + ((C::fragment(e, j) * PY + q) * 64 + lane) * 16) = pf[q];
      }
    }
  };
  if constexpr (L == 64) {
    products(wave, true);
    products(3 - wave, false);
  } else {
    products(wave & 1, wave < 2);
  }
  __syncthreads();   // K and Q have been read: the inverse takes their place
  if (wave < TT && lane < 16) {
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
  for (int d = 1; d < TT; ++d) {
    if (wave < TT - d) {
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
  for (int e = 0; e < TT; ++e)
#pragma unroll
    for (int j = 0; j <= e / 2; ++j) {
      const int f = C::fragment(e, j);
      if (f % 4 != wave) continue;
      const int t = 16 * e + n16;
      u32x4 tf[kPieces];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int s = 32 * j + 16 * u + 4 * g;
        const f32x4 v = *reinterpret_cast<const f32x4*>(&lds_t[t * LD + s]);
        const f32x4 b = *reinterpret_cast<const f32x4*>(&lds_beta[s]);
        float w[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) w[r] = s + r <= t ? v[r] * b[r] : 0.f;   // (above the diagonal nothing is written)
        uint32_t lo[kPieces], hi[kPieces];
        split_pair<kPieces>(w[0], w[1], lo);
        split_pair<kPieces>(w[2], w[3], hi);
#pragma unroll
        for (int q = 0; q < kPieces; ++q) tf[q][2 * u] = lo[q], tf[q][2 * u + 1] = hi[q];
      }
#pragma unroll
      for (int q = 0; q < kPieces; ++q) *reinterpret_cast<u32x4*>(blob + C::kT + ((f * kPieces + q) * 64 + lane) * 16) = tf[q];
    }
}

// 16 bytes a lane from memory to LDS, at `lds` (uniform over the wavefront) + 16 lane;
// offsets outside the buffer give zeros. The compiler does not know of these loads:
// arrived() waits for all of a wavefront's. (m0 is the compiler's for single
// instructions only, none of which are used here.)
__device__ __forceinline__ void load_lds(const i32x4& buffer, uint32_t offset, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(__builtin_amdgcn_readfirstlane((int)lds)), "v"(offset), "s"(buffer)
               : "memory");
}
__device__ __forceinline__ void arrived() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

__device__ __forceinline__ i32x4 buffer_of(const void* base, uint32_t bytes) {
  const uint64_t p = reinterpret_cast<uint64_t>(base);
  i32x4 r;
  r[0] = __builtin_amdgcn_readfirstlane((int)(uint32_t)p);
  r[1] = __builtin_amdgcn_readfirstlane((int)(uint32_t)(p >> 32) & 0xFFFF);
  r[2] = __builtin_amdgcn_readfirstlane((int)bytes);
  r[3] = 0x00020000;
  return r;
}

__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)reinterpret_cast<uintptr_t>((const __attribute__((address_space(3))) uint8_t*)p);
}

// A workgroup owns 16 WV columns of one head's state, a wavefront 16 of them and all
// of d_k, in registers over the whole sequence. Rows k of the state are spread over
// the lanes so that a lane's 8 of a step of 32 follow one another, in the order in
// which a product takes 8 rows of K: state register [kt][r] of lane group g is row
// 32 (kt / 2) + 8 g + 4 (kt & 1) + r. Results of one product are then factors of the
// next as they are, S of K S, X of T X, U of P U and K^T U, and nothing but the inputs
// passes through LDS, which holds two chunks' (one on its way from memory).
template <typename T, int DK, int L, int PI, int PY, int WV>
__global__ __launch_bounds__(64 * WV) void delta_kernel(DeltaArgs a) {
  typedef Tile<DK> TB;
  typedef Chunk<L, PY> C;
  constexpr int TT = C::kTiles, KT = DK / 16, KS = DK / 32, TS = L / 32;
  constexpr int BB = L * TB::kBytes, KEYS = 2 * PI * BB;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2][KEYS + C::kBytes];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n16 = lane & 15, g = lane >> 4;
  // Workgroups go round the 8 XCDs: those of one head and sequence, which read the
  // same chunks, go to one XCD's cache.
  const int id = blockIdx.x >> 3;
  const int unit = id / a.vblocks * 8 + (blockIdx.x & 7);
  if (unit >= a.units) return;
  const int v0 = (id % a.vblocks) * 16 * WV;
  const int h = unit % a.l.H, sq = unit / a.l.H, hk = h / a.l.per_key;
  const int dk = a.l.dk, dv = a.l.dv;
  int begin, len;
  const int slot0 = __builtin_amdgcn_readfirstlane(first_slot<L>(a.l.s, sq, begin, len));
  begin = __builtin_amdgcn_readfirstlane(begin), len = __builtin_amdgcn_readfirstlane(len);
  const int chunks = (len + L - 1) / L;
  if (chunks == 0 && a.l.state_in) return;

  const int sv = v0 + 16 * wave + n16;
  float* const st = a.l.state + ((size_t)sq * a.l.H + h) * dk * dv + sv;
  auto state_row = [&](int kt, int r) { return 32 * (kt >> 1) + 8 * g + 4 * (kt & 1) + r; };
  f32x4 S[KT];
#pragma unroll
  for (int kt = 0; kt < KT; ++kt) {
    S[kt] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (a.l.state_in) {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (state_row(kt, r) < dk && sv < dv) S[kt][r] = st[(size_t)state_row(kt, r) * dv];
    }
  }

  const T* const kp = reinterpret_cast<const T*>(a.l.k) + begin * a.l.k_stride + (size_t)hk * dk;
  const T* const qp = reinterpret_cast<const T*>(a.l.q) + begin * a.l.q_stride + (size_t)hk * dk;
  const T* const vp = reinterpret_cast<const T*>(a.l.v) + begin * a.l.v_stride + (size_t)h * dv;
  T* const op = reinterpret_cast<T*>(a.l.o) + begin * a.l.o_stride + (size_t)h * dv;
  const int krow = (int)(a.l.k_stride * sizeof(T)), qrow = (int)(a.l.q_stride * sizeof(T));
  const int vrow = (int)(a.l.v_stride * sizeof(T)), orow = (int)(a.l.o_stride * sizeof(T));

  // ---- a chunk's K, Q (fp32: their pieces), T, P and decays to LDS
  auto fetch = [&](int c) {
    const uint32_t to = lds_address(lds[c & 1]);
    if constexpr (PI == 1) {
      const int rows = min(len - c * L, L);
      const i32x4 rK = buffer_of(kp + (int64_t)c * L * a.l.k_stride, (uint32_t)(rows * krow));
      const i32x4 rQ = buffer_of(qp + (int64_t)c * L * a.l.q_stride, (uint32_t)(rows * qrow));
#pragma unroll
      for (int i0 = 0; i0 < BB / 1024; i0 += WV) {
        const int i = i0 + wave;
        if (BB / 1024 % WV != 0 && i >= BB / 1024) break;
        // LDS holds a row's pieces in Tile's order
        const int row = (64 * i + lane) / (DK / 8), at = (64 * i + lane) % (DK / 8);
        const int piece = (int)(TB::at(row, at) - row * TB::kBytes) >> 4;
        const bool in = piece * 8 < dk;
        load_lds(rK, in ? (uint32_t)(row * krow + piece * 16) : kOutside, to + i * 1024);
        load_lds(rQ, in ? (uint32_t)(row * qrow + piece * 16) : kOutside, to + BB + i * 1024);
      }
    } else {
      const i32x4 r = buffer_of(a.keys + ((size_t)(slot0 + c) * (a.l.H / a.l.per_key) + hk) * KEYS, KEYS);
#pragma unroll
      for (int i0 = 0; i0 < KEYS / 1024; i0 += WV) {
        const int i = i0 + wave;
        if (KEYS / 1024 % WV != 0 && i >= KEYS / 1024) break;
        load_lds(r, (uint32_t)(i * 1024 + lane * 16), to + i * 1024);
      }
    }
    const i32x4 r = buffer_of(a.chunks + ((size_t)(slot0 + c) * a.l.H + h) * C::kBytes, C::kBytes);
#pragma unroll
    for (int i0 = 0; i0 < C::kBytes / 1024; i0 += WV) {
      const int i = i0 + wave;
      if (C::kBytes / 1024 % WV != 0 && i >= C::kBytes / 1024) break;
      load_lds(r, (uint32_t)(i * 1024 + lane * 16), to + KEYS + i * 1024);
    }
  };
  uint32_t vn[TT][4];   // v of tokens 16 e + 4 g + r, this lane's column
  uint32_t voff = sv < dv ? (uint32_t)(4 * g * vrow + sv * (int)sizeof(T)) : kOutside;
  auto fetch_v = [&](int c) {
    const ChunkRows<L> rV(vp, vrow, c * L, len);
#pragma unroll
    for (int e = 0; e < TT; ++e)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int at = (int)(voff + (uint32_t)((16 * e + r) * vrow));
        if constexpr (PI == 1) vn[e][r] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(rV.rsrc, at, 0, 0) << 16;
        else vn[e][r] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(rV.rsrc, at, 0, 0);
      }
  };
  const uint32_t a_frag = TB::fragment(lane);
  const uint32_t a_tr = TB::at(4 * g + (n16 >> 2), n16 & 3);
  const uint32_t ooff = v0 + 16 * wave + 4 * g < dv ? (uint32_t)(n16 * orow + (v0 + 16 * wave + 4 * g) * (int)sizeof(T)) : kOutside;

  if (chunks > 0) {
    fetch(0);
    fetch_v(0);
  }
  for (int c = 0; c < chunks; ++c) {
    arrived();
    __syncthreads();   // this chunk is in LDS, and the last one has been read
    if (c + 1 < chunks) fetch(c + 1);
    const uint8_t* const lds_k = lds[c & 1];
    const uint8_t* const lds_q = lds_k + PI * BB;
    const uint8_t* const blob = lds_k + KEYS;
    const float* const gates = reinterpret_cast<const float*>(blob + C::kGates);
    local(voff);

    // ---- K S0 (rows t, columns v) and S0^T Q^T (rows v, columns t)
    f32x4 x[TT], o[TT];
#pragma unroll
    for (int e = 0; e < TT; ++e) x[e] = o[e] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < KS; ++i) {
      u32x4 sf[kPieces];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t lo[kPieces], hi[kPieces];
        split_pair<kPieces>(S[2 * i + u][0], S[2 * i + u][1], lo);
        split_pair<kPieces>(S[2 * i + u][2], S[2 * i + u][3], hi);
#pragma unroll
        for (int q = 0; q < kPieces; ++q) sf[q][2 * u] = lo[q], sf[q][2 * u + 1] = hi[q];
      }
#pragma unroll
      for (int p = 0; p < PI; ++p)
#pragma unroll
        for (int e = 0; e < TT; ++e) {
          const u32x4 kf = *reinterpret_cast<const u32x4*>(lds_k + p * BB + 16 * e * TB::kBytes + (a_frag ^ (i << 6)));
          const u32x4 qf = *reinterpret_cast<const u32x4*>(lds_q + p * BB + 16 * e * TB::kBytes + (a_frag ^ (i << 6)));
#pragma unroll
          for (int q = 0; q < kPieces; ++q)
            if (p + q < 3) x[e] = mfma(kf, sf[q], x[e]);
#pragma unroll
          for (int q = 0; q < PY; ++q)
            if (p + q < 3) o[e] = mfma(sf[q], qf, o[e]);
        }
    }
    settle();
    // ---- X = V - e^c K S0
    uint32_t odd = 0;
#pragma unroll
    for (int e = 0; e < TT; ++e) {
      const f32x4 to = *reinterpret_cast<const f32x4*>(gates + C::kTo + 16 * e + 4 * g);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        x[e][r] = __builtin_fmaf(-to[r], x[e][r], __uint_as_float(vn[e][r]));
        odd |= (__float_as_uint(x[e][r]) & 0x7F800000u) + 0x00800000u;
      }
    }
    if (c + 1 < chunks) fetch_v(c + 1);
    // A product takes all tokens, with weights of zero for later ones: an X that is not
    // finite is taken out, and its column NaN from its token on
    int bad = reinterpret_cast<const int*>(gates)[C::kBad];
    const bool any = __builtin_amdgcn_ballot_w64((odd & 0x80000000u) != 0 || bad < L) != 0;
    if (any) {
#pragma unroll
      for (int e = 0; e < TT; ++e)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if ((__float_as_uint(x[e][r]) & 0x7F800000u) == 0x7F800000u) bad = min(bad, 16 * e + 4 * g + r);
      bad = min(bad, __shfl_xor(bad, 16, 64));
      bad = min(bad, __shfl_xor(bad, 32, 64));
#pragma unroll
      for (int e = 0; e < TT; ++e)
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (16 * e + 4 * g + r >= bad) x[e][r] = 0.f;
    }
    // ---- U = T X
    u32x4 xf[TS][kPieces];
#pragma unroll
    for (int e = 0; e < TT; ++e) {
      uint32_t lo[kPieces], hi[kPieces];
      split_pair<kPieces>(x[e][0], x[e][1], lo);
      split_pair<kPieces>(x[e][2], x[e][3], hi);
#pragma unroll
      for (int q = 0; q < kPieces; ++q) xf[e / 2][q][2 * (e & 1)] = lo[q], xf[e / 2][q][2 * (e & 1) + 1] = hi[q];
    }
    f32x4 u[TT];
#pragma unroll
    for (int e = 0; e < TT; ++e) u[e] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < TS; ++j)
#pragma unroll
      for (int p = 0; p < kPieces; ++p)
#pragma unroll
        for (int e = 2 * j; e < TT; ++e) {
          const u32x4 tf = *reinterpret_cast<const u32x4*>(blob + C::kT + ((C::fragment(e, j) * kPieces + p) * 64 + lane) * 16);
#pragma unroll
          for (int q = 0; q < kPieces; ++q)
            if (p + q < 3) u[e] = mfma(tf, xf[j][q], u[e]);
        }
    settle();
    // ---- O^T = e^c S0^T Q^T + U^T P^T
    {
      u32x4 uf[TS][PY];
#pragma unroll
      for (int e = 0; e < TT; ++e) {
        uint32_t lo[PY], hi[PY];
        split_pair<PY>(u[e][0], u[e][1], lo);
        split_pair<PY>(u[e][2], u[e][3], hi);
#pragma unroll
        for (int q = 0; q < PY; ++q) uf[e / 2][q][2 * (e & 1)] = lo[q], uf[e / 2][q][2 * (e & 1) + 1] = hi[q];
        const float to = gates[C::kTo + 16 * e + n16];
#pragma unroll
        for (int r = 0; r < 4; ++r) o[e][r] *= to;
      }
#pragma unroll
      for (int j = 0; j < TS; ++j)
#pragma unroll
        for (int p = 0; p < PY; ++p)
#pragma unroll
          for (int e = 2 * j; e < TT; ++e) {
            const u32x4 pf = *reinterpret_cast<const u32x4*>(blob + C::kP + ((C::fragment(e, j) * PY + p) * 64 + lane) * 16);
#pragma unroll
            for (int q = 0; q < PY; ++q)
              if (p + q < PY) o[e] = mfma(uf[j][q], pf, o[e]);
          }
    }
    // ---- S <- e^{c_n} S0 + K^T (e^{c_n - c} U)
    u32x4 wf[TS][kPieces];
#pragma unroll
    for (int e = 0; e < TT; ++e) {
      const f32x4 from = *reinterpret_cast<const f32x4*>(gates + C::kFrom + 16 * e + 4 * g);
      uint32_t lo[kPieces], hi[kPieces];
      split_pair<kPieces>(u[e][0] * from[0], u[e][1] * from[1], lo);
      split_pair<kPieces>(u[e][2] * from[2], u[e][3] * from[3], hi);
#pragma unroll
      for (int q = 0; q < kPieces; ++q) wf[e / 2][q][2 * (e & 1)] = lo[q], wf[e / 2][q][2 * (e & 1) + 1] = hi[q];
    }
    const float decay = gates[C::kDecay];
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
#pragma unroll
      for (int r = 0; r < 4; ++r) S[kt][r] *= decay;
#pragma unroll
      for (int j = 0; j < TS; ++j)
#pragma unroll
        for (int p = 0; p < PI; ++p) {
          const u32x4 kf = read_tr8<DK>(lds_k + p * BB + 32 * j * TB::kBytes + (a_tr ^ ((kt >> 1) << 6)) + 8 * (kt & 1));
#pragma unroll
          for (int q = 0; q < kPieces; ++q)
            if (p + q < 3) S[kt] = mfma(kf, wf[j][q], S[kt]);
        }
    }
    settle();
    if (any) {
      if (bad < L) {
#pragma unroll
        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
          for (int r = 0; r < 4; ++r) S[kt][r] = __builtin_nanf("");
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int from = __shfl(bad, 4 * g + r, 64);
#pragma unroll
        for (int e = 0; e < TT; ++e)
          if (16 * e + n16 >= from) o[e][r] = __builtin_nanf("");
      }
    }
    const ChunkRows<L> rO(op, orow, c * L, len);
#pragma unroll
    for (int e = 0; e < TT; ++e) {
      const int at = (int)(ooff + (uint32_t)(16 * e * orow));
      if constexpr (PI == 1)
        __builtin_amdgcn_raw_buffer_store_b64(u32x2{bf16_pair(o[e][0], o[e][1]), bf16_pair(o[e][2], o[e][3])}, rO.rsrc, at, 0, 0);
      else
        __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, o[e]), rO.rsrc, at, 0, 0);
    }
  }
#pragma unroll
  for (int kt = 0; kt < KT; ++kt)
#pragma unroll
    for (int r = 0; r < 4; ++r)
      if (state_row(kt, r) < dk && sv < dv) st[(size_t)state_row(kt, r) * dv] = S[kt][r];
}

typedef void (*DeltaFn)(DeltaArgs);

struct DeltaPlan {
  int L, waves;
  DeltaFn prepare, scan;
  int64_t slots, units, vblocks;
  size_t chunk_bytes, bytes;
};

template <typename T, int DK, int L, int PI, int PY>
void pick_delta(DeltaPlan& w, const rsq_linear_attn* p) {
  w.L = L;
  w.prepare = delta_prepare_kernel<T, DK, L, PI, PY>;
  const int64_t tiles = ceil_div(p->d_v, 16);
  w.units = (int64_t)p->seqs * p->heads;
  w.waves = tiles > 4 && w.units >= 128 ? 8 : tiles > 2 && w.units * ceil_div(tiles, 4) >= 64 ? 4 : 1;
  w.scan = w.waves == 8 ? delta_kernel<T, DK, L, PI, PY, 8> : w.waves == 4 ? delta_kernel<T, DK, L, PI, PY, 4>
                                                                           : delta_kernel<T, DK, L, PI, PY, 1>;
  w.vblocks = ceil_div(tiles, w.waves);
  // a sequence of len rows has ceil(len / L) chunks; with their rows apart, at most tokens / L + seqs in all
  w.slots = p->tokens / L + p->seqs;
  w.chunk_bytes = (size_t)w.slots * p->heads * Chunk<L, PY>::kBytes;
  w.bytes = w.chunk_bytes + (PI > 1 ? (size_t)w.slots * p->key_heads * 2 * PI * L * DK * 2 : 0);
}

rsq_status plan_delta(const rsq_linear_attn* p, DeltaPlan& w) {
  if (p->dtype == RSQ_BF16) {
    if (p->d_k <= 64) pick_delta<Bf16, 64, 64, 1, 2>(w, p);
    else if (p->d_k <= 128) pick_delta<Bf16, 128, 64, 1, 2>(w, p);
    else pick_delta<Bf16, 256, 32, 1, 2>(w, p);
  } else {
    if (p->d_k <= 64) pick_delta<float, 64, 32, 3, 3>(w, p);
    else pick_delta<float, 128, 32, 3, 3>(w, p);
  }
  if (const rsq_status s = check_blocks(w.slots * p->heads, 256)) return s;
  return check_blocks(ceil_div(w.units, 8) * 8 * w.vblocks, 64 * w.waves);
}

}  // namespace

rsq_status delta_workspace(const rsq_linear_attn* p, size_t* bytes) {
  DeltaPlan w;
  if (const rsq_status s = plan_delta(p, w)) return s;
  *bytes = p->max_len > 0 ? w.bytes : 0;
  return RSQ_OK;
}

rsq_status run_delta(const rsq_linear_attn* p, const LinearArgs& l, void* stream) {
  DeltaPlan w;
  if (const rsq_status s = plan_delta(p, w)) return s;
  if (p->max_len > 0) {
    if (!p->workspace || !aligned(p->workspace, 16)) return fail(RSQ_E_INVALID, "workspace is NULL or not 16-byte aligned");
    if (p->workspace_bytes < w.bytes)
      return fail(RSQ_E_BUFFER, "workspace has %zu bytes, the call needs %zu", p->workspace_bytes, w.bytes);
  }
  DeltaArgs a{};
  a.l = l;
  a.chunks = static_cast<uint8_t*>(p->workspace);
  a.keys = a.chunks + w.chunk_bytes;
  a.slots = (int32_t)w.slots, a.vblocks = (int32_t)w.vblocks, a.units = (int32_t)w.units;
  if (p->max_len > 0) {
    hipLaunchKernelGGL(w.prepare, dim3((unsigned)(w.slots * p->heads)), dim3(256), 0, (hipStream_t)stream, a);
    if (const rsq_status s = launched("delta rule, chunks")) return s;
  }
  const int64_t blocks = ceil_div(w.units, 8) * 8 * w.vblocks;
  hipLaunchKernelGGL(w.scan, dim3((unsigned)blocks), dim3(64 * w.waves), 0, (hipStream_t)stream, a);
  return launched("delta rule");
}

}  // namespace rsq

// Selective state-space scan of prompts (ssm.hpp has the recurrence), in chunks
// of kL tokens. With c_t the sum of d A over a chunk's tokens up to t, S0 the
// state before the chunk and L its last token, the recurrence unrolls to
//   y_t = e^{c_t} S0^T C_t + sum_{s <= t} P_ts x_s + D x_t,
//   P_ts = e^{c_t - c_s} d_s (C_t . B_s),
//   S   <- e^{c_L} S0 + sum_s B_s (d_s e^{c_L - c_s} x_s)^T:
// four small matrix products a chunk, on the matrix cores.
//
// Bytes and products would take 57 and 27 us of 16384 tokens (64 heads of 128 x
// 64, bf16, 283 MB); it takes 226 to 235 (by the card; 1.2 TB/s, 185 TFLOP/s counting
// the recurrence's own 5 operations an element). What that goes to: the state is
// formed twice (first for the segments' starts, a third of the time, then along with
// y), from three bf16 pieces each (two would make errors of 2e-6 of an exact fp32
// state), and it and the token weights enter y as two pieces. In the second pass the
// vector unit (splitting, weighting, rounding and the diagonal's mask) is busy for 55%
// of the cycles, LDS for 47 and the matrix cores for 31, which three wavefronts a
// SIMD between four barriers a chunk overlap little; registers (168) and LDS (43.5
// KB) keep a fourth out. Measured without gain: C B^T made once for all heads of a
// group, decays of four chunks at a time by four wavefronts (5% longer), raised
// priority for the products, remainders by dot products, more of the segments' states
// on their way at once, P in LDS of its own (one barrier less), C laid out for wider
// reads.
// 333 fp32 tokens take 19 us, 9 of them two empty launches.
#include <initializer_list>

#include "chunk.hpp"
#include "host_util.hpp"
#include "ssm.hpp"

namespace rsq {
namespace {

constexpr int kL = 64;        // tokens of a chunk
constexpr int kV = 64;        // state columns of a workgroup
constexpr int kThreads = 256;
constexpr int kWide = 1 << 30;   // no power of two
typedef ChunkRows<kL> Rows;

struct ScanArgs {
  SsmArgs s;
  float* ws_state;    // [heads][column blocks][slots][DK / 16][256] float4
  float* ws_decay;    // [heads][slots]: log2 of a segment's decay
  int32_t vblocks;    // column blocks of kV
  int32_t segs;       // segments of the longest sequence
  int32_t seg_chunks; // chunks of a segment
  int32_t slots;      // segments of all sequences that are cut into two and more
  const float* alpha; // decays themselves (linear attention), NULL for 1
  int64_t alpha_stride;   // 0: one row for all tokens
};

// What a workgroup scans: a segment of a sequence that is cut into `used` of them,
// or a whole one (used 1).
struct Share {
  int seq, seg, used;
  int slot;         // of the sequence's first segment
  int begin, len;   // the sequence's rows (counted in 31 bits)
};

__device__ __forceinline__ void read_sequence(const ScanArgs& a, int s, int& begin, int& len) {
  int64_t n;
  begin = (int)seq_range(a.s.q, s, n);
  len = (int)n;
}

// segments of a sequence, none if it is not cut
__device__ __forceinline__ int cut_segments(const ScanArgs& a, int len) {
  const int chunks = (len + kL - 1) / kL;
  const int used = (chunks + a.seg_chunks - 1) / a.seg_chunks;
  return used > 1 ? used : 0;
}

// Units of work: the segments of the sequences that are cut, in the sequences'
// order (a unit's number is its slot in the workspace), then every sequence once,
// for those that are not. Where the offsets fall, sequences overlap and may have
// more segments than the workspace has slots: the ones that do not fit are scanned
// whole. False for a unit without work. The wavefronts all find the same, each
// for itself: 64 sequences at a time, with the sequences before to be counted
// only where a sequence is cut.
__device__ __forceinline__ bool find_share(const ScanArgs& a, int unit, int lane, Share& f) {
  if (!a.s.q.offsets) {
    f.used = a.segs;
    f.seq = unit / a.segs;
    f.slot = f.seq * a.segs;
    f.seg = unit - f.slot;
    read_sequence(a, f.seq, f.begin, f.len);
    return true;
  }
  const bool whole = unit >= a.slots;
  const int own = unit - a.slots, seqs = a.s.q.seqs;
  f = Share{own, 0, 1, 0, 0, 0};
  if (whole) {
    read_sequence(a, own, f.begin, f.len);
    f.begin = __builtin_amdgcn_readfirstlane(f.begin), f.len = __builtin_amdgcn_readfirstlane(f.len);
    if (cut_segments(a, f.len) == 0) return true;
  }
  int first = 0;   // slots of the sequences before these 64
  for (int s0 = 0; s0 < seqs && first <= a.slots; s0 += 64) {
    const int s = s0 + lane;
    int begin = 0, len = 0;
    if (s < seqs) read_sequence(a, s, begin, len);
    const int n = cut_segments(a, len);
    const int upto = (int)wave_scan((double)n);
    const uint64_t hit = __builtin_amdgcn_ballot_w64(whole ? s == own : unit < first + upto);
    if (hit) {
      const int l = __builtin_ctzll(hit);
      const int end = first + __builtin_amdgcn_readlane(upto, l);
      if (whole) return end > a.slots;
      f.used = __builtin_amdgcn_readlane(n, l);
      f.seq = s0 + l;
      f.slot = end - f.used;
      f.seg = unit - f.slot;
      f.begin = __builtin_amdgcn_readlane(begin, l), f.len = __builtin_amdgcn_readlane(len, l);
      return end <= a.slots;
    }
    first += __builtin_amdgcn_readlane(upto, 63);
  }
  return whole;
}

// PI pieces of the inputs, PY of the computed factors of y (P and S), 3 of the
// weighted x that enters the state (a state stays exact to fp32). Products of
// pieces below 2^-24 are left out. bf16 outputs take PY = 2: y before its own
// rounding is then off by 2^-16 of its terms. (One piece would leave 2^-8 of them,
// as much as that rounding where the state makes up y; it took 205 us where two take
// 235, 16384 tokens of 64 heads of 128 x 64.)
//
// Shares of the four wavefronts: wavefront w owns the 16 columns 16 w of the state
// and of y, and all of d_k, in registers over the whole segment; S enters y straight
// from them. Of P it makes the rows of the 16 tokens 16 w (w + 1 tiles), which pass
// through LDS, in C's place. Wavefront 0, with the fewest tiles of P, works out the
// next chunk's decays. STATES: only the state is wanted (a
// segment before the last, scanned first so that the segments can run side by
// side).
// ALPHA: the decays are given (linear attention: x is v, B is k and C is q, the
// token weights are 1), for every token or once for all of a head. 8192 tokens in 8
// sequences, 16 heads of 128 x 128, one decay a head (150 MB: 30 us), take 89 us for
// the same products and splitting as the scan.
template <typename T, int DK, int PI, int PY, bool STATES, bool ALPHA>
__global__ __launch_bounds__(kThreads, PI > 1 ? (DK > 64 ? 1 : 2) : DK > 128 ? 2 : 3) void scan_kernel(ScanArgs a) {
  constexpr int PW = 3;
  constexpr int KT = DK / 16, KS = DK / 32;
  typedef Tile<DK> TB;
  typedef Tile<kV> TX;
  constexpr int BB = kL * TB::kBytes, XB = kL * TX::kBytes;   // bytes of a piece's tile
  __shared__ __attribute__((aligned(16))) uint8_t lds_b[PI * BB];
  __shared__ __attribute__((aligned(16))) uint8_t lds_x[PI * XB];
  // C, and once that has been read, P's pieces as products take them: [tokens / 16][s / 32][piece][lane]
  constexpr int PB = kL / 16 * (kL / 32) * PY * 1024;
  __shared__ __attribute__((aligned(16))) uint8_t lds_c[STATES ? 16 : PI * BB > PB ? PI * BB : PB];
  // of a chunk's tokens, by the chunk's parity: d_t e^{c_L - c_t}, and the factors of e^{c_t - c_s}
  constexpr int LY = STATES ? 4 : kL;
  __shared__ __attribute__((aligned(16))) float lds_w[2][kL], lds_from[2][LY], lds_to[2][LY];
  __shared__ __attribute__((aligned(16))) int lds_whole[2][LY];
  __shared__ float lds_decay[2];     // e^{c_L}
  __shared__ int lds_mid[2];         // the power of two that is shifted, or kWide for none
  __shared__ int lds_first[2][kV];   // first token of a column whose x is not finite
  __shared__ int lds_bad[2];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n16 = lane & 15, g = lane >> 4;
  int id = blockIdx.x;
  const int h = id % a.s.H;
  id /= a.s.H;
  const int vb = id % a.vblocks;
  id /= a.vblocks;
  const float A2 = ALPHA ? 0.f : a.s.A[h] * 1.44269504088896f;   // decays in powers of two
  const float gamma = ALPHA && a.alpha && a.alpha_stride == 0 ? a.alpha[h] : 1.f;
  const float Dh = a.s.D ? a.s.D[h] : 0.f;
  const float dt_bias = a.s.dt_bias ? a.s.dt_bias[h] : 0.f;
  Share share;
  if (!find_share(a, id, lane, share)) return;
  // (all uniform over the workgroup, which the compiler cannot know of loaded offsets)
  const int sq = __builtin_amdgcn_readfirstlane(share.seq), seg = __builtin_amdgcn_readfirstlane(share.seg);
  const int used = __builtin_amdgcn_readfirstlane(share.used), slot0 = __builtin_amdgcn_readfirstlane(share.slot);
  const int64_t begin = __builtin_amdgcn_readfirstlane(share.begin);
  const int len = __builtin_amdgcn_readfirstlane(share.len);
  const int dk = a.s.dk, dv = a.s.dv, v0 = vb * kV;
  const int chunks = (len + kL - 1) / kL;
  // the first pass covers the segments before the last; the second all of them
  if (STATES ? seg == used - 1 : chunks == 0 && a.s.state_in) return;

  // ---- the state before the segment
  f32x4 S[KT];   // S[kt][r] = state[16 kt + 4 g + r][v0 + 16 wave + n16]
  const int sv = v0 + 16 * wave + n16;
  float* st = a.s.state + ((size_t)sq * a.s.H + h) * dk * dv + sv;
  const size_t slot = (size_t)KT * kThreads;
  f32x4* ws = reinterpret_cast<f32x4*>(a.ws_state) + (((size_t)h * a.vblocks + vb) * a.slots + slot0) * slot + tid;
  float* wd = a.ws_decay + (size_t)h * a.slots + slot0;
#pragma unroll
  for (int kt = 0; kt < KT; ++kt) S[kt] = f32x4{0.f, 0.f, 0.f, 0.f};
  const bool split = used > 1;
  if (seg == 0 && a.s.state_in && (STATES || !split)) {
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int k = 16 * kt + 4 * g + r;
        if (k < dk && sv < dv) S[kt][r] = st[(size_t)k * dv];
      }
  }
  if constexpr (STATES) {
    // the second pass writes the final state over the initial one: keep it in
    // the last segment's slot, which no segment's own state takes
    if (seg == 0)
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) ws[(size_t)(used - 1) * slot + kt * kThreads] = S[kt];
  } else if (split) {
    // slot 0 holds the state after segment 0, slot j > 0 what segment j adds
    const size_t first = seg == 0 ? used - 1 : 0;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) S[kt] = ws[first * slot + kt * kThreads];
    // (the next segment's state is on its way while one is added)
    f32x4 add[KT];
    if (seg > 1)
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) add[kt] = ws[slot + kt * kThreads];
    for (int j = 1; j < seg; ++j) {
      const float e = __builtin_amdgcn_exp2f(wd[j]);
      f32x4 now[KT];
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) now[kt] = add[kt];
      if (j + 1 < seg)
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) add[kt] = ws[(j + 1) * slot + kt * kThreads];
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int r = 0; r < 4; ++r) S[kt][r] = __builtin_fmaf(S[kt][r], e, now[kt][r]);
    }
  }

  const T* x = reinterpret_cast<const T*>(a.s.x) + begin * a.s.x_stride + (size_t)h * dv + v0;
  const T* Bp = reinterpret_cast<const T*>(a.s.B) + begin * a.s.b_stride + (size_t)(h / a.s.per_group) * dk;
  const T* Cp = reinterpret_cast<const T*>(a.s.C) + begin * a.s.c_stride + (size_t)(h / a.s.per_group) * dk;
  T* y = reinterpret_cast<T*>(a.s.y) + begin * a.s.y_stride + (size_t)h * dv + v0;
  const int xrow = (int)(a.s.x_stride * sizeof(T)), brow = (int)(a.s.b_stride * sizeof(T));
  const int crow = (int)(a.s.c_stride * sizeof(T)), yrow = (int)(a.s.y_stride * sizeof(T));

  // ---- a chunk's rows: B, C and x go through registers to LDS one chunk ahead
  constexpr int NB = kL * (DK / 8) / kThreads, RB = kThreads / (DK / 8);   // loads a thread, rows of one load
  constexpr int NX = kL * (kV / 8) / kThreads, RX = kThreads / (kV / 8);
  Vec8<T, PI> rb[NB], rx[NX], rc[STATES ? 1 : NB];
  const int bk = (tid % (DK / 8)) * 8, xv8 = (tid % (kV / 8)) * 8;
  uint32_t boff = bk < dk ? (uint32_t)(tid / (DK / 8) * brow + bk * (int)sizeof(T)) : kOutside;
  uint32_t xoff = v0 + xv8 < dv ? (uint32_t)(tid / (kV / 8) * xrow + xv8 * (int)sizeof(T)) : kOutside;
  const int c_end = split ? min(chunks, (seg + 1) * a.seg_chunks) : chunks;
  const int end = min(len, c_end * kL);   // (int: c_end * kL is below len + kL)
  auto load_bx = [&](int t0) {
    const Rows rB(Bp, brow, t0, end), rX(x, xrow, t0, end);
#pragma unroll
    for (int i = 0; i < NB; ++i) rb[i].load(rB, boff + (uint32_t)(i * RB * brow));
#pragma unroll
    for (int i = 0; i < NX; ++i) rx[i].load(rX, xoff + (uint32_t)(i * RX * xrow));
  };
  uint32_t coff = bk < dk ? (uint32_t)(tid / (DK / 8) * crow + bk * (int)sizeof(T)) : kOutside;
  auto load_c = [&](int t0) {
    const Rows rC(Cp, crow, t0, end);
#pragma unroll
    for (int i = 0; i < (STATES ? 0 : NB); ++i) rc[i].load(rC, coff + (uint32_t)(i * RB * crow));
  };
  // a load of fewer than 16 rows (d_k = 256: 8) moves f by the bits of row 8
  auto flip = [](int rows) { return (uint32_t)((rows >> 3) & 1 ? 9 << 4 : 0); };
  uint32_t yoff = (uint32_t)(n16 * yrow + (16 * wave + 4 * g) * (int)sizeof(T));
  // LDS addresses of this lane
  uint32_t a_bput = TB::at(tid / (DK / 8), tid % (DK / 8)), a_xput = TX::at(tid / (kV / 8), tid % (kV / 8));
  uint32_t a_frag = TB::fragment(lane), a_btr = TB::transposed(lane), a_xtr = TX::transposed(lane);
  uint32_t a_four = TB::four(n16, lane), a_xown = TX::four(n16, lane);
  // Running sums of the log2 decays, in 64 bits: differences of them are small
  // next to the sums where decays are strong. A row past the sequence neither
  // decays nor adds.
  double total = 0.0;
  auto decays = [&](float dt, int t0, int par) {
    float delta = 0.f;
    double cum = 0.;   // (not 0 A: A may be infinite)
    if (t0 + lane < len) {
      if constexpr (ALPHA) {
        delta = 1.f;
        cum = log2((double)(a.alpha_stride ? dt : gamma));
      } else {
        delta = dt + dt_bias;
        if (a.s.softplus) delta = softplus(delta);
        cum = (double)delta * (double)A2;
      }
    }
    // a token that decays by 2^-2000 keeps nothing of an fp32 state
    cum = cum < -2000. ? -2000. : cum > 2000. ? 2000. : cum;
    cum = wave_scan(cum);
    const double last = lane63(cum);
    total += last;
    lds_w[par][lane] = __builtin_amdgcn_exp2f((float)(last - cum)) * delta;
    if (lane == 0) lds_decay[par] = __builtin_amdgcn_exp2f((float)last);
    if constexpr (!STATES) {
      // c = n + f with n whole: 2^{c_t - c_s} = 2^{f_t} 2^{n_t - n_s} 2^{-f_s}.
      // Where the n are within kNear of their middle, powers of two shift them
      // into the factors of t and s; both ways give the same bits.
      constexpr int kNear = 40;
      const double n = rint(cum);
      const float f = (float)(cum - n);
      const int whole = (int)n, mid = (int)rint(0.5 * last);
      const bool narrow = __builtin_amdgcn_ballot_w64(!(fabs(cum - 0.5 * last) < kNear)) == 0;
      const int shift = narrow ? mid - whole : 0;
      lds_from[par][lane] = __builtin_amdgcn_ldexpf(__builtin_amdgcn_exp2f(-f) * delta, shift);
      lds_to[par][lane] = __builtin_amdgcn_ldexpf(__builtin_amdgcn_exp2f(f), -shift);
      lds_whole[par][lane] = whole;
      if (lane == 0) lds_mid[par] = narrow ? mid : kWide;
    }
  };
  const void* dtp = reinterpret_cast<const T*>(a.s.dt) + begin * a.s.dt_stride + h;
  int dtrow = (int)(a.s.dt_stride * sizeof(T));
  if constexpr (ALPHA) dtp = a.alpha + begin * a.alpha_stride + h, dtrow = (int)(a.alpha_stride * 4);
  auto load_dt = [&](int t0) {
    const Rows r(dtp, dtrow, t0, end);   // (no bytes where one row is for all tokens)
    if constexpr (PI == 1 && !ALPHA) return (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(r.rsrc, lane * dtrow, 0, 0) << 16;
    else return (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(r.rsrc, lane * dtrow, 0, 0);
  };

  int c = seg * a.seg_chunks;
  uint32_t dt_next = 0u;   // dt of the chunk after this one (of use to wavefront 0)
  if (c < c_end) {
    const uint32_t dt = load_dt(c * kL);
    dt_next = load_dt((c + 1) * kL);
    load_bx(c * kL);
    load_c(c * kL);
    if (wave == 0) decays(__uint_as_float(dt), c * kL, c & 1);
  }
  if (tid < 2 * kV) lds_first[tid / kV][tid % kV] = kL;
  if (tid < 2) lds_bad[tid] = 0;
  __syncthreads();
  for (; c < c_end; ++c) {
    const int t0 = c * kL;
    const int par = c & 1;
    local(boff), local(xoff), local(coff), local(yoff), local(a_bput), local(a_xput), local(a_frag), local(a_btr);
    local(a_xtr), local(a_four), local(a_xown);
    // ---- stage: inputs to LDS
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      u32x4 p[PI];
      rb[i].pieces(p);
#pragma unroll
      for (int q = 0; q < PI; ++q) *reinterpret_cast<u32x4*>(lds_b + q * BB + i * RB * TB::kBytes + (a_bput ^ flip(i * RB))) = p[q];
    }
#pragma unroll
    for (int i = 0; i < NX; ++i) {
      u32x4 p[PI];
      rx[i].pieces(p);
#pragma unroll
      for (int q = 0; q < PI; ++q) *reinterpret_cast<u32x4*>(lds_x + q * XB + i * RX * TX::kBytes + a_xput) = p[q];
    }
    // A product with x_s takes every s of a chunk, weights of later tokens
    // being zero: an infinity or a NaN there would reach earlier tokens. It is
    // taken out, and its column is NaN from its token on.
    uint32_t odd = 0;
#pragma unroll
    for (int i = 0; i < NX; ++i) odd |= rx[i].bad_bits();
    if (odd & (PI == 1 ? 0x80008000u : 0x80000000u)) {
#pragma unroll
      for (int i = 0; i < NX; ++i) {
        Vec8<T, PI> v = rx[i];
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (v.bad(e)) {
            v.clear(e);
            atomicMin(&lds_first[par][xv8 + e], tid / (kV / 8) + i * RX);
          }
        u32x4 p[PI];
        v.pieces(p);
#pragma unroll
        for (int q = 0; q < PI; ++q) *reinterpret_cast<u32x4*>(lds_x + q * XB + i * RX * TX::kBytes + a_xput) = p[q];
      }
      lds_bad[par] = 1;
    }
    if constexpr (!STATES) {
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        u32x4 p[PI];
        rc[i].pieces(p);
#pragma unroll
        for (int q = 0; q < PI; ++q) *reinterpret_cast<u32x4*>(lds_c + q * BB + i * RB * TB::kBytes + (a_bput ^ flip(i * RB))) = p[q];
      }
    }
    __syncthreads();
    const bool bad = __builtin_amdgcn_readfirstlane(lds_bad[par]) != 0;
    const bool more = c + 1 < c_end;
    const uint32_t dt = dt_next;
    dt_next = load_dt(t0 + 2 * kL);
    load_bx(t0 + kL);
    if (wave == 0 && more) decays(__uint_as_float(dt), t0 + kL, par ^ 1);
    if (tid < kV) lds_first[par ^ 1][tid] = kL;
    if (tid == kV) lds_bad[par ^ 1] = 0;

    if constexpr (!STATES) {
      // ---- S^T C, 16 tokens a tile: the lane's rows of S, in fours of 32 keys, are the product's
      f32x4 sc[kL / 16];
#pragma unroll
      for (int e = 0; e < kL / 16; ++e) sc[e] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        u32x4 sf[PY];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t lo[PY], hi[PY];
          split_pair<PY>(S[2 * i + e][0], S[2 * i + e][1], lo);
          split_pair<PY>(S[2 * i + e][2], S[2 * i + e][3], hi);
#pragma unroll
          for (int q = 0; q < PY; ++q) sf[q][2 * e] = lo[q], sf[q][2 * e + 1] = hi[q];
        }
#pragma unroll
        for (int p = 0; p < PI; ++p)
#pragma unroll
          for (int e = 0; e < kL / 16; ++e) {
            const uint8_t* at = lds_c + p * BB + 16 * e * TB::kBytes;
            const u32x2 c0 = *reinterpret_cast<const u32x2*>(at + (a_four ^ ((2 * i) << 5)));
            const u32x2 c1 = *reinterpret_cast<const u32x2*>(at + (a_four ^ ((2 * i + 1) << 5)));
            const u32x4 c = {c0[0], c0[1], c1[0], c1[1]};
#pragma unroll
            for (int q = 0; q < PY; ++q)
              if (p + q < 3) sc[e] = mfma(sf[q], c, sc[e]);
          }
        __builtin_amdgcn_sched_barrier(0);
      }
      settle();
      u32x4 cf[KS][PI];
#pragma unroll
      for (int i = 0; i < KS; ++i)
#pragma unroll
        for (int p = 0; p < PI; ++p)
          cf[i][p] = *reinterpret_cast<const u32x4*>(lds_c + p * BB + 16 * wave * TB::kBytes + (a_frag ^ (i << 6)));
      const int tt = 16 * wave + n16;   // this lane's token
      const int mid = __builtin_amdgcn_readfirstlane(lds_mid[par]);
      __builtin_amdgcn_sched_barrier(0);
      const float to = lds_to[par][tt];
      const int power = mid == kWide ? lds_whole[par][tt] : mid;
      u32x4 pf[kL / 32][PY];
      // ---- P^T (rows s, columns t), two tiles (a k-step of y) at a time, up to
      // the diagonal's; two chains of dependent products run side by side
#pragma unroll
      for (int j2 = 0; j2 < kL / 32; ++j2) {
        if (2 * j2 <= wave) {
          f32x4 acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
          for (int i = 0; i < KS; ++i)
#pragma unroll
            for (int p = 0; p < PI; ++p)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const u32x4 bf = *reinterpret_cast<const u32x4*>(lds_b + p * BB + (32 * j2 + 16 * e) * TB::kBytes +
                                                                 (a_frag ^ (i << 6)));
#pragma unroll
                for (int q = 0; q < PI; ++q)
                  if (p + q < 3) acc[e] = mfma(bf, cf[i][q], acc[e]);
              }
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int s0 = 32 * j2 + 16 * e;
            const f32x4 from = *reinterpret_cast<const f32x4*>(&lds_from[par][s0 + 4 * g]);
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[e][r] *= from[r] * to;   // (one factor may be 2^40 where the other is 2^-40)
            if (mid == kWide) {
              const i32x4 n = *reinterpret_cast<const i32x4*>(&lds_whole[par][s0 + 4 * g]);
#pragma unroll
              for (int r = 0; r < 4; ++r) acc[e][r] = __builtin_amdgcn_ldexpf(acc[e][r], power - n[r]);
            }
            if (2 * j2 + 1 >= wave) {   // later tokens: out, whatever their weight
#pragma unroll
              for (int r = 0; r < 4; ++r) acc[e][r] = s0 + 4 * g + r <= tt ? acc[e][r] : 0.f;
            }
            uint32_t lo[PY], hi[PY];
            split_pair<PY>(acc[e][0], acc[e][1], lo);
            split_pair<PY>(acc[e][2], acc[e][3], hi);
#pragma unroll
            for (int q = 0; q < PY; ++q) pf[j2][q][2 * e] = lo[q], pf[j2][q][2 * e + 1] = hi[q];
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      auto at_p = [&](int tile, int j2, int q) { return lds_c + (((tile * (kL / 32) + j2) * PY + q) * 64 + lane) * 16; };
      __syncthreads();   // C has been read
#pragma unroll
      for (int j2 = 0; j2 < kL / 32; ++j2)
        if (2 * j2 <= wave) {
#pragma unroll
          for (int q = 0; q < PY; ++q) *reinterpret_cast<u32x4*>(at_p(wave, j2, q)) = pf[j2][q];
        }
      __syncthreads();   // P is there
      // ---- y^T (rows v, columns t), this wavefront's 16 columns
      u32x4 xf[kL / 32][PI];
#pragma unroll
      for (int j2 = 0; j2 < kL / 32; ++j2)
#pragma unroll
        for (int p = 0; p < PI; ++p) xf[j2][p] = read_tr8<kV>(lds_x + p * XB + 32 * j2 * TX::kBytes + (a_xtr ^ (wave << 5)));
      const Rows rY(y, yrow, t0, len);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int e = 0; e < kL / 16; ++e) {
        // e^{c_t} of the tokens
        const float before = __builtin_amdgcn_ldexpf(lds_to[par][16 * e + n16], mid == kWide ? lds_whole[par][16 * e + n16] : mid);
#pragma unroll
        for (int r = 0; r < 4; ++r) sc[e][r] *= before;
      }
#pragma unroll
      for (int j2 = 0; j2 < kL / 32; ++j2)
#pragma unroll
        for (int q = 0; q < PY; ++q)
#pragma unroll
          for (int e = 2 * j2; e < kL / 16; ++e) {
            const u32x4 pt = *reinterpret_cast<const u32x4*>(at_p(e, j2, q));
#pragma unroll
            for (int p = 0; p < PI; ++p)
              if (p + q < 3) sc[e] = mfma(xf[j2][p], pt, sc[e]);
          }
      settle();
#pragma unroll
      for (int e = 0; e < kL / 16; ++e) {
        // D x, from the pieces of x (their sum is exact)
        float xv[4];
#pragma unroll
        for (int p = PI - 1; p >= 0; --p) {
          const u32x2 w = *reinterpret_cast<const u32x2*>(lds_x + p * XB + 16 * e * TX::kBytes + (a_xown ^ (wave << 5)));
          const float part[4] = {low_half(w[0]), high_half(w[0]), low_half(w[1]), high_half(w[1])};
#pragma unroll
          for (int r = 0; r < 4; ++r) xv[r] = p == PI - 1 ? part[r] : xv[r] + part[r];
        }
        float out[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) out[r] = __builtin_fmaf(Dh, xv[r], sc[e][r]);
        if (bad) {
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (16 * e + n16 >= lds_first[par][16 * wave + 4 * g + r]) out[r] = __builtin_nanf("");
        }
        const uint32_t at = yoff + (uint32_t)(16 * e * yrow);
        auto store = [&](uint32_t at) {
          if constexpr (PI == 1)
            __builtin_amdgcn_raw_buffer_store_b64(u32x2{bf16_pair(out[0], out[1]), bf16_pair(out[2], out[3])}, rY.rsrc, (int)at, 0, 0);
          else
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, f32x4{out[0], out[1], out[2], out[3]}), rY.rsrc, (int)at, 0, 0);
        };
        if (v0 + kV <= dv) store(at);
        else store(v0 + 16 * wave + 4 * g < dv ? at : kOutside);
      }
      load_c(t0 + kL);
    }

    // (the state after a segment is the next segment's own to work out)
    if (STATES || c + 1 < c_end || seg == used - 1) {
      // ---- S <- decay S + B^T (w x)
      const float decay = lds_decay[par];
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int r = 0; r < 4; ++r) S[kt][r] *= decay;
      // Two tiles of keys side by side; the next two are read while they are worked on.
      constexpr int STEPS = KT / 2 * PI;
      u32x4 bf[2][2];
      auto read_b = [&](int ts, int step, u32x4 (&out)[2]) {
        const int k2 = step / PI * 2, p = step % PI;
#pragma unroll
        for (int e = 0; e < 2; ++e) out[e] = read_tr8<DK>(lds_b + p * BB + 32 * ts * TB::kBytes + (a_btr ^ ((k2 + e) << 5)));
      };
      read_b(0, 0, bf[0]);
#pragma unroll
      for (int ts = 0; ts < kL / 32; ++ts) {
        u32x4 xr[PI];
#pragma unroll
        for (int p = 0; p < PI; ++p) xr[p] = read_tr8<kV>(lds_x + p * XB + 32 * ts * TX::kBytes + (a_xtr ^ (wave << 5)));
        const f32x4 w0 = *reinterpret_cast<const f32x4*>(&lds_w[par][32 * ts + 4 * g]);
        const f32x4 w1 = *reinterpret_cast<const f32x4*>(&lds_w[par][32 * ts + 16 + 4 * g]);
        u32x4 xw[PW];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float lo = low_half(xr[PI - 1][i]), hi = high_half(xr[PI - 1][i]);
#pragma unroll
          for (int p = PI - 2; p >= 0; --p) lo += low_half(xr[p][i]), hi += high_half(xr[p][i]);
          lo *= i < 2 ? w0[2 * i] : w1[2 * i - 4];
          hi *= i < 2 ? w0[2 * i + 1] : w1[2 * i - 3];
          uint32_t p3[PW];
          split_pair<PW>(lo, hi, p3);
#pragma unroll
          for (int q = 0; q < PW; ++q) xw[q][i] = p3[q];
        }
#pragma unroll
        for (int step = 0; step < STEPS; ++step) {
          const int now = (ts * STEPS + step) & 1;
          if (step + 1 < STEPS) read_b(ts, step + 1, bf[now ^ 1]);
          else if (ts + 1 < kL / 32) read_b(ts + 1, 0, bf[now ^ 1]);
          __builtin_amdgcn_sched_barrier(0);
#pragma unroll
          for (int q = 0; q < PW; ++q)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (step % PI + q < 3) S[step / PI * 2 + e] = mfma(bf[now][e], xw[q], S[step / PI * 2 + e]);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      settle();
      if (bad) {
        if (lds_first[par][16 * wave + n16] < kL) {
#pragma unroll
          for (int kt = 0; kt < KT; ++kt)
#pragma unroll
            for (int r = 0; r < 4; ++r) S[kt][r] = __builtin_nanf("");
        }
      }
    }
    __syncthreads();   // the chunk's LDS has been read
  }

  // ---- the state after the segment
  if constexpr (STATES) {
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) ws[(size_t)seg * slot + kt * kThreads] = S[kt];
    if (tid == 0 && vb == 0) wd[seg] = (float)total;
  } else if (seg == used - 1) {
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int k = 16 * kt + 4 * g + r;
        if (k < dk && sv < dv) st[(size_t)k * dv] = S[kt][r];
      }
  }
}

}  // namespace
}  // namespace rsq

namespace rsq {
namespace {

typedef void (*ScanFn)(ScanArgs);

template <bool STATES, bool ALPHA>
ScanFn pick_scan(bool bf16, int dkp) {
  if (bf16) {
    switch (dkp) {
      case 64: return scan_kernel<Bf16, 64, 1, 2, STATES, ALPHA>;
      case 128: return scan_kernel<Bf16, 128, 1, 2, STATES, ALPHA>;
      default: return scan_kernel<Bf16, 256, 1, 2, STATES, ALPHA>;
    }
  }
  return dkp == 64 ? scan_kernel<float, 64, 3, 3, STATES, ALPHA> : scan_kernel<float, 128, 3, 3, STATES, ALPHA>;
}

struct ScanPlan {
  int dkp, vblocks, segs, seg_chunks, slots;
  int64_t state_blocks, blocks;   // of the first and of the second pass
  size_t state_bytes, bytes;
};

// Sequences are cut into segments that run side by side when heads and
// sequences alone do not fill the chip: about `target` workgroups of equal
// length, three for each of 256 compute units (16384 tokens of 64 heads of 128 x 64
// bf16 235 us, with 512 254, with 1024 251), or two where d_k lets no third in (8192
// tokens of 64 heads of 256 x 64 bf16 198 us, with 768 222, with 256 286; of 16 heads
// of 128 x 128 fp32 201, 230, 216).
// A segment costs its chunks one and a half times (the states first), and one
// step for each segment before it, about 1/7 of a chunk's time: with n chunks,
// sqrt(n / 11) of them a segment is the shortest that pays, and two chunks are
// not worth a second pass.
//
// Of packed sequences only the longest is known here. With their rows apart, a
// sequence of len rows has at most (len - 1) / (64 per) segments after its first, so
// all have at most tokens / (64 per), and the sequences that are cut are at most as
// many: one prompt of 16384 tokens beside 255 of one (64 heads of 128 x 64 bf16)
// needs 25 MB and 16768 workgroups, where a slot for each sequence's longest would
// take 3.2 GB and 98304.
rsq_status plan_scan(const rsq_ssm* p, ScanPlan& w) {
  w.dkp = p->d_k <= 64 ? 64 : p->d_k <= 128 ? 128 : 256;
  w.vblocks = (int)ceil_div(p->d_v, kV);
  const int64_t base = (int64_t)p->heads * w.vblocks;
  const int64_t longest = ceil_div(p->max_len, kL);
  int64_t total = ceil_div(p->tokens, kL) + p->seqs;
  if (total > longest * p->seqs) total = longest * p->seqs;
  const int64_t target = w.dkp > (p->dtype == RSQ_BF16 ? 128 : 64) ? 512 : 768;
  int64_t per = ceil_div(total * base, target);
  while (per * per * 11 < longest) ++per;
  if (per > longest || longest < 3) per = longest > 0 ? longest : 1;
  w.segs = (int)(longest > 0 ? ceil_div(longest, per) : 1);
  w.seg_chunks = (int)per;
  int64_t slots = w.segs > 1 ? (int64_t)p->seqs * w.segs : 0;
  if (p->offsets) {
    const int64_t more = p->tokens / (kL * per);
    const int64_t most = more + (more < p->seqs ? more : p->seqs);
    if (slots > most) slots = most;
  }
  w.state_blocks = base * slots;
  w.blocks = base * (p->offsets || w.segs == 1 ? slots + p->seqs : slots);
  if (const rsq_status s = check_blocks(w.blocks, kThreads)) return s;
  w.slots = (int)slots;
  w.state_bytes = (size_t)w.state_blocks * (w.dkp / 16) * kThreads * 16;
  w.bytes = w.state_bytes + (size_t)p->heads * slots * 4;
  return RSQ_OK;
}

rsq_status check_scan_workspace(const rsq_ssm* p, const ScanPlan& w) {
  if (!w.bytes) return RSQ_OK;
  if (!p->workspace || !aligned(p->workspace, 16)) return fail(RSQ_E_INVALID, "workspace is NULL or not 16-byte aligned");
  if (p->workspace_bytes < w.bytes)
    return fail(RSQ_E_BUFFER, "workspace has %zu bytes, the scan needs %zu", p->workspace_bytes, w.bytes);
  return RSQ_OK;
}

rsq_status launch_scan(const rsq_ssm* p, const ScanPlan& w, const float* alpha, int64_t alpha_stride, bool gated, void* stream) {
  ScanArgs a{};
  a.s = ssm_args(p);
  a.ws_state = static_cast<float*>(p->workspace);
  a.ws_decay = reinterpret_cast<float*>(static_cast<uint8_t*>(p->workspace) + w.state_bytes);
  a.vblocks = w.vblocks, a.segs = w.segs, a.seg_chunks = w.seg_chunks, a.slots = w.slots;
  a.alpha = alpha, a.alpha_stride = alpha ? alpha_stride : 0;
  const bool bf16 = p->dtype == RSQ_BF16;
  if (w.slots > 0) {
    const ScanFn fn = gated ? pick_scan<true, true>(bf16, w.dkp) : pick_scan<true, false>(bf16, w.dkp);
    hipLaunchKernelGGL(fn, dim3((unsigned)w.state_blocks), dim3(kThreads), 0, (hipStream_t)stream, a);
    if (const rsq_status s = launched("selective scan, segment states")) return s;
  }
  const ScanFn fn = gated ? pick_scan<false, true>(bf16, w.dkp) : pick_scan<false, false>(bf16, w.dkp);
  hipLaunchKernelGGL(fn, dim3((unsigned)w.blocks), dim3(kThreads), 0, (hipStream_t)stream, a);
  return launched("selective scan");
}

}  // namespace

rsq_status decayed_scan_workspace(const rsq_ssm* p, size_t* bytes) {
  ScanPlan w;
  if (const rsq_status s = plan_scan(p, w)) return s;
  *bytes = w.bytes;
  return RSQ_OK;
}

rsq_status run_decayed_scan(const rsq_ssm* p, const float* alpha, int64_t alpha_stride, void* stream) {
  ScanPlan w;
  if (const rsq_status s = plan_scan(p, w)) return s;
  if (const rsq_status s = check_scan_workspace(p, w)) return s;
  return launch_scan(p, w, alpha, alpha_stride, true, stream);
}

}  // namespace rsq

using namespace rsq;

extern "C" rsq_status rsq_ssm_scan_workspace(const rsq_ssm* p, size_t* bytes) {
  if (!bytes) return fail(RSQ_E_INVALID, "bytes is NULL");
  if (const rsq_status s = check_ssm(p, true)) return s;
  ScanPlan w;
  if (const rsq_status s = plan_scan(p, w)) return s;
  *bytes = w.bytes;
  return RSQ_OK;
}

extern "C" rsq_status rsq_ssm_scan(const rsq_ssm* p, void* stream) {
  if (const rsq_status s = check_ssm(p, true)) return s;
  if (!p->state) return fail(RSQ_E_INVALID, "state is NULL");
  const int64_t size = p->dtype == RSQ_BF16 ? 2 : 4;
  // (the kernel counts rows in int, some chunks ahead of the last)
  if (p->max_len > 0x7fffffff - 4096) return fail(RSQ_E_UNSUPPORTED, "max_len %lld", (long long)p->max_len);
  for (const int64_t stride : {p->x_stride, p->b_stride, p->c_stride, p->dt_stride, p->y_stride})
    if (stride > kMaxRowBytes / size)
      return fail(RSQ_E_UNSUPPORTED, "rows %lld elements apart, more than 2^24 bytes", (long long)stride);
  if (const rsq_status s = check_ssm_memory(p)) return s;
  ScanPlan w;
  if (const rsq_status s = plan_scan(p, w)) return s;
  if (const rsq_status s = check_scan_workspace(p, w)) return s;
  return launch_scan(p, w, nullptr, 0, false, stream);
}

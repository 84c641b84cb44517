// Selective state-space scan of prompts (ssm.hpp has the recurrence), in chunks
// of kL tokens. With c_t the sum of d A over a chunk's tokens up to t, S0 the
// state before the chunk and L its last token, the recurrence unrolls to
//   y_t = e^{c_t} S0^T C_t + sum_{s <= t} P_ts x_s + D x_t,
//   P_ts = e^{c_t - c_s} d_s (C_t . B_s),
//   S   <- e^{c_L} S0 + sum_s B_s (d_s e^{c_L - c_s} x_s)^T:
// four small matrix products a chunk, on the matrix cores.
#include "host_util.hpp"
#include "ssm.hpp"

namespace rsq {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kL = 64;        // tokens of a chunk
constexpr int kV = 64;        // state columns of a workgroup
constexpr int kThreads = 256;
constexpr int kPad = 8;       // elements behind each LDS row: rows start 16 bytes apart in the banks

struct ScanArgs {
  SsmArgs s;
  float* ws_state;    // [seqs][heads][column blocks][segments][DK / 16][256] float4
  float* ws_decay;    // [seqs][heads][segments]: log2 of a segment's decay
  int32_t vblocks;    // column blocks of kV
  int32_t segs;       // segments of the longest sequence
  int32_t seg_chunks; // chunks of a segment
};

__device__ __forceinline__ f32x4 mfma(const u32x4& a, const u32x4& b, const f32x4& c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// the high halves of two floats as a bf16 pair (a in the low half)
__device__ __forceinline__ uint32_t high_pair(float a, float b) {
  return __builtin_amdgcn_perm(__float_as_uint(b), __float_as_uint(a), 0x07060302u);
}

// An fp32 value as N bf16 pieces. One piece is rounded to nearest-even (2^-9
// relative). Three pieces hold all 24 bits: each takes the leading 8 of what
// is left, so the products of pieces are exact and their sum is rounded in
// fp32 only.
template <int N>
__device__ __forceinline__ void split_pair(float a, float b, uint32_t (&p)[N]) {
  if constexpr (N == 1) {
    p[0] = bf16_pair(a, b);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      p[i] = high_pair(a, b);
      a -= __uint_as_float(__float_as_uint(a) & 0xFFFF0000u);
      b -= __uint_as_float(__float_as_uint(b) & 0xFFFF0000u);
    }
  }
}

// 8 consecutive input elements as PI pieces of 4 words each
template <typename T, int PI>
struct Vec8 {
  u32x4 raw[PI == 1 ? 1 : 2];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (auto& r : raw) r = u32x4{0u, 0u, 0u, 0u};
  }
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (PI == 1 ? 1 : 2); ++i) raw[i] = reinterpret_cast<const u32x4*>(p)[i];
  }
  __device__ __forceinline__ void pieces(u32x4 (&out)[PI]) const {
    if constexpr (PI == 1) {
      out[0] = raw[0];
    } else {
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t p[PI];
        split_pair<PI>(__uint_as_float(raw[w >> 1][2 * (w & 1)]), __uint_as_float(raw[w >> 1][2 * (w & 1) + 1]), p);
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
  __device__ __forceinline__ bool any_bad() const {
    bool b = false;
#pragma unroll
    for (int e = 0; e < 8; ++e) b = b || bad(e);
    return b;
  }
};

typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// Transposed read: rows r0 .. r0 + 3 of 16 columns from c0 on, where r0 is the
// 16-lane group's; lane i of the group gets the four rows' elements of column
// c0 + i. (ds_read_b64_tr_b16: lane i names the i-th run of four elements.)
__device__ __forceinline__ u32x2 read_tr(const uint16_t* base, int stride, int r0, int c0, int lane) {
  const int i = lane & 15;
  const uint16_t* p = base + (r0 + (i >> 2)) * stride + c0 + 4 * (i & 3);
  return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)p));
}

// Contraction index of a k-step of 32 over tokens: lane group g holds tokens
// 4g .. 4g + 3 and 16 + 4g .. 16 + 4g + 3. A product's lanes hold its rows in
// fours like this, so P leaves one product and enters the next in registers.
__device__ __forceinline__ u32x4 read_tr8(const uint16_t* base, int stride, int r0, int c0, int lane) {
  const int g = lane >> 4;
  const u32x2 lo = read_tr(base, stride, r0 + 4 * g, c0, lane);
  const u32x2 hi = read_tr(base, stride, r0 + 16 + 4 * g, c0, lane);
  return u32x4{lo[0], lo[1], hi[0], hi[1]};
}

// PI pieces of the inputs, PY of the computed factors of y (P and S), 3 of the
// weighted x that enters the state (a state stays exact to fp32). Products of
// pieces below 2^-24 are left out.
//
// Shares of the four wavefronts: for y, wavefront w owns the 16 tokens 16 w;
// for the state, the 16 columns 16 w and all of d_k, in registers over the
// whole segment. STATES: only the state is wanted (a segment before the last,
// scanned first so that the segments can run side by side).
template <typename T, int DK, int PI, int PY, bool STATES>
__global__ __launch_bounds__(kThreads, DK > 128 || PI > 1 ? 1 : 2) void scan_kernel(ScanArgs a) {
  constexpr int PW = 3;
  constexpr int KT = DK / 16, KS = DK / 32;
  constexpr int SK = DK + kPad, SV = kV + kPad;
  __shared__ __attribute__((aligned(16))) uint16_t lds_b[PI][kL][SK];
  __shared__ __attribute__((aligned(16))) uint16_t lds_x[PI][kL][SV];
  __shared__ __attribute__((aligned(16))) uint16_t lds_s[STATES ? 1 : PY][STATES ? 1 : kV][SK];   // S^T: [column][key]
  __shared__ __attribute__((aligned(16))) float lds_hi[kL], lds_lo[kL], lds_d[kL], lds_w[kL];
  __shared__ int lds_first[2][kV];   // first token of a column whose x is not finite
  __shared__ int lds_bad[2];

  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int n16 = lane & 15, g = lane >> 4;
  int id = blockIdx.x;
  const int h = id % a.s.H;
  id /= a.s.H;
  const int vb = id % a.vblocks;
  id /= a.vblocks;
  const int seg = id % a.segs;
  const int sq = id / a.segs;
  int64_t len;
  const int64_t begin = seq_range(a.s.q, sq, len);
  const int dk = a.s.dk, dv = a.s.dv, v0 = vb * kV;
  const int64_t chunks = (len + kL - 1) / kL;
  const int used = (int)((chunks + a.seg_chunks - 1) / a.seg_chunks);
  // the first pass covers the segments before the last; the second all of them
  if (STATES ? seg >= used - 1 : seg >= used && (seg > 0 || a.s.state_in)) return;

  // ---- the state before the segment
  f32x4 S[KT];   // S[kt][r] = state[16 kt + 4 g + r][v0 + 16 wave + n16]
  const int sv = v0 + 16 * wave + n16;
  float* st = a.s.state + ((size_t)sq * a.s.H + h) * dk * dv + sv;
  const size_t slot = (size_t)KT * kThreads;
  f32x4* ws = reinterpret_cast<f32x4*>(a.ws_state) + (((size_t)sq * a.s.H + h) * a.vblocks + vb) * a.segs * slot + tid;
  float* wd = a.ws_decay + ((size_t)sq * a.s.H + h) * a.segs;
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
      for (int kt = 0; kt < KT; ++kt) ws[(size_t)(a.segs - 1) * slot + kt * kThreads] = S[kt];
  } else if (split) {
    // slot 0 holds the state after segment 0, slot j > 0 what segment j adds
    const size_t first = seg == 0 ? a.segs - 1 : 0;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) S[kt] = ws[first * slot + kt * kThreads];
    for (int j = 1; j < seg; ++j) {
      const float e = __builtin_amdgcn_exp2f(wd[j]);
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) {
        const f32x4 t = ws[j * slot + kt * kThreads];
#pragma unroll
        for (int r = 0; r < 4; ++r) S[kt][r] = __builtin_fmaf(S[kt][r], e, t[r]);
      }
    }
  }

  const T* x = reinterpret_cast<const T*>(a.s.x) + begin * a.s.x_stride + (size_t)h * dv + v0;
  const T* Bp = reinterpret_cast<const T*>(a.s.B) + begin * a.s.b_stride + (size_t)(h / a.s.per_group) * dk;
  const T* Cp = reinterpret_cast<const T*>(a.s.C) + begin * a.s.c_stride + (size_t)(h / a.s.per_group) * dk;
  T* y = reinterpret_cast<T*>(a.s.y) + begin * a.s.y_stride + (size_t)h * dv + v0;
  const float A2 = a.s.A[h] * 1.44269504088896f;   // decays in powers of two
  const float Dh = a.s.D ? a.s.D[h] : 0.f;

  // ---- a chunk's rows, loaded one chunk ahead
  constexpr int NB = kL * (DK / 8) / kThreads;
  constexpr int NX = kL * (kV / 8) / kThreads;
  Vec8<T, PI> rb[NB], rx[NX], rc[KS];
  float delta = 0.f;
  auto load = [&](int64_t t0) {
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int u = tid + kThreads * i, k = (u % (DK / 8)) * 8;
      const int64_t t = t0 + u / (DK / 8);
      rb[i].zero();
      if (t < len && k < dk) rb[i].load(Bp + t * a.s.b_stride + k);
    }
#pragma unroll
    for (int i = 0; i < NX; ++i) {
      const int u = tid + kThreads * i, v = (u % (kV / 8)) * 8;
      const int64_t t = t0 + u / (kV / 8);
      rx[i].zero();
      if (t < len && v0 + v < dv) rx[i].load(x + t * a.s.x_stride + v);
    }
    if constexpr (!STATES) {
      const int64_t t = t0 + 16 * wave + n16;
#pragma unroll
      for (int i = 0; i < KS; ++i) {
        const int k = 32 * i + 8 * g;
        rc[i].zero();
        if (t < len && k < dk) rc[i].load(Cp + t * a.s.c_stride + k);
      }
    }
    // a row past the sequence neither decays nor adds
    delta = t0 + lane < len ? ssm_delta<T>(a.s, begin + t0 + lane, h) : 0.f;
  };

  const int64_t c_end = chunks < (int64_t)(seg + 1) * a.seg_chunks ? chunks : (int64_t)(seg + 1) * a.seg_chunks;
  int64_t c = (int64_t)seg * a.seg_chunks;
  double total = 0.0;
  if (c < c_end) load(c * kL);
  if (tid < 2 * kV) lds_first[tid / kV][tid % kV] = kL;
  if (tid < 2) lds_bad[tid] = 0;
  __syncthreads();
  for (; c < c_end; ++c) {
    const int64_t t0 = c * kL;
    const int par = (int)(c & 1);
    // ---- stage: inputs and the state to LDS, the decays
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int u = tid + kThreads * i;
      u32x4 p[PI];
      rb[i].pieces(p);
#pragma unroll
      for (int q = 0; q < PI; ++q) *reinterpret_cast<u32x4*>(&lds_b[q][u / (DK / 8)][(u % (DK / 8)) * 8]) = p[q];
    }
#pragma unroll
    for (int i = 0; i < NX; ++i) {
      const int u = tid + kThreads * i, row = u / (kV / 8), v = (u % (kV / 8)) * 8;
      // A product with x_s takes every s of a chunk, weights of later tokens
      // being zero: an infinity or a NaN there would reach earlier tokens. It
      // is taken out, and its column is NaN from its token on.
      if (rx[i].any_bad()) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (rx[i].bad(e)) {
            rx[i].clear(e);
            atomicMin(&lds_first[par][v + e], row);
          }
        lds_bad[par] = 1;
      }
      u32x4 p[PI];
      rx[i].pieces(p);
#pragma unroll
      for (int q = 0; q < PI; ++q) *reinterpret_cast<u32x4*>(&lds_x[q][row][v]) = p[q];
    }
    if constexpr (!STATES) {
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) {
        uint32_t lo[PY], hi[PY];
        split_pair<PY>(S[kt][0], S[kt][1], lo);
        split_pair<PY>(S[kt][2], S[kt][3], hi);
#pragma unroll
        for (int q = 0; q < PY; ++q)
          *reinterpret_cast<u32x2*>(&lds_s[q][16 * wave + n16][16 * kt + 4 * g]) = u32x2{lo[q], hi[q]};
      }
    }
    // running sums of the log2 decays, in 64 bits: differences of them are
    // small next to the sums where decays are strong
    double cum = (double)delta * (double)A2;
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) {
      const double o = __shfl_up(cum, m, 64);
      if (lane >= m) cum += o;
    }
    const double last = __shfl(cum, 63, 64);
    const float decay = __builtin_amdgcn_exp2f((float)last);
    total += last;
    if (wave == 0) {
      const float hi = (float)cum;
      lds_hi[lane] = hi;
      lds_lo[lane] = (float)(cum - (double)hi);
      lds_d[lane] = delta;
      lds_w[lane] = __builtin_amdgcn_exp2f((float)(last - cum)) * delta;
    }
    u32x4 cf[STATES ? 1 : KS][PI];
    if constexpr (!STATES) {
#pragma unroll
      for (int i = 0; i < KS; ++i) rc[i].pieces(cf[i]);
    }
    __syncthreads();
    const bool bad = lds_bad[par] != 0;
    if (c + 1 < c_end) load(t0 + kL);
    if (tid < kV) lds_first[par ^ 1][tid] = kL;
    if (tid == kV) lds_bad[par ^ 1] = 0;

    if constexpr (!STATES) {
      const int tt = 16 * wave + n16;   // this lane's token
      const float chi = lds_hi[tt], clo = lds_lo[tt];
      // ---- P^T (rows s, columns t), two tiles of s a k-step, up to the diagonal
      u32x4 pf[2][PY];
#pragma unroll
      for (int st2 = 0; st2 < 2; ++st2) {
        if (2 * st2 > wave) break;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int s0 = 32 * st2 + 16 * half;
          f32x4 acc = {0.f, 0.f, 0.f, 0.f};
          if (s0 <= 16 * wave) {
#pragma unroll
            for (int i = 0; i < KS; ++i)
#pragma unroll
              for (int p = 0; p < PI; ++p) {
                const u32x4 bf = *reinterpret_cast<const u32x4*>(&lds_b[p][s0 + n16][32 * i + 8 * g]);
#pragma unroll
                for (int q = 0; q < PI; ++q)
                  if (p + q < 3) acc = mfma(bf, cf[i][q], acc);
              }
          }
          const f32x4 shi = *reinterpret_cast<const f32x4*>(&lds_hi[s0 + 4 * g]);
          const f32x4 slo = *reinterpret_cast<const f32x4*>(&lds_lo[s0 + 4 * g]);
          const f32x4 sd = *reinterpret_cast<const f32x4*>(&lds_d[s0 + 4 * g]);
          float pv[4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float e = __builtin_amdgcn_exp2f((chi - shi[r]) + (clo - slo[r]));
            pv[r] = s0 + 4 * g + r <= tt ? acc[r] * (e * sd[r]) : 0.f;
          }
          uint32_t lo[PY], hi[PY];
          split_pair<PY>(pv[0], pv[1], lo);
          split_pair<PY>(pv[2], pv[3], hi);
#pragma unroll
          for (int q = 0; q < PY; ++q) pf[st2][q][2 * half] = lo[q], pf[st2][q][2 * half + 1] = hi[q];
        }
      }
      // ---- y^T (rows v, columns t)
      const float et = __builtin_amdgcn_exp2f(chi + clo);
#pragma unroll
      for (int vt = 0; vt < kV / 16; ++vt) {
        f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < KS; ++i)
#pragma unroll
          for (int p = 0; p < PY; ++p) {
            const u32x4 sf = *reinterpret_cast<const u32x4*>(&lds_s[p][16 * vt + n16][32 * i + 8 * g]);
#pragma unroll
            for (int q = 0; q < PI; ++q)
              if (p + q < 3) acc = mfma(sf, cf[i][q], acc);
          }
#pragma unroll
        for (int r = 0; r < 4; ++r) acc[r] *= et;
#pragma unroll
        for (int st2 = 0; st2 < 2; ++st2) {
          if (2 * st2 > wave) break;
#pragma unroll
          for (int p = 0; p < PI; ++p) {
            const u32x4 xf = read_tr8(&lds_x[p][0][0], SV, 32 * st2, 16 * vt, lane);
#pragma unroll
            for (int q = 0; q < PY; ++q)
              if (p + q < 3) acc = mfma(xf, pf[st2][q], acc);
          }
        }
        // D x, from the pieces of x (their sum is exact)
        float xv[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int p = PI - 1; p >= 0; --p) {
          const u32x2 w = *reinterpret_cast<const u32x2*>(&lds_x[p][tt][16 * vt + 4 * g]);
          xv[0] += __uint_as_float(w[0] << 16), xv[1] += __uint_as_float(w[0] & 0xFFFF0000u);
          xv[2] += __uint_as_float(w[1] << 16), xv[3] += __uint_as_float(w[1] & 0xFFFF0000u);
        }
        float out[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          out[r] = __builtin_fmaf(Dh, xv[r], acc[r]);
          if (bad && tt >= lds_first[par][16 * vt + 4 * g + r]) out[r] = __builtin_nanf("");
        }
        const int v = 16 * vt + 4 * g;
        if (t0 + tt < len && v0 + v < dv) {
          T* yp = y + (t0 + tt) * a.s.y_stride + v;
          if constexpr (PI == 1) *reinterpret_cast<u32x2*>(yp) = u32x2{bf16_pair(out[0], out[1]), bf16_pair(out[2], out[3])};
          else *reinterpret_cast<f32x4*>(yp) = f32x4{out[0], out[1], out[2], out[3]};
        }
      }
    }

    // ---- S <- decay S + B^T (w x)
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int r = 0; r < 4; ++r) S[kt][r] *= decay;
#pragma unroll
    for (int ts = 0; ts < kL / 32; ++ts) {
      u32x4 xr[PI];
#pragma unroll
      for (int p = 0; p < PI; ++p) xr[p] = read_tr8(&lds_x[p][0][0], SV, 32 * ts, 16 * wave, lane);
      const f32x4 w0 = *reinterpret_cast<const f32x4*>(&lds_w[32 * ts + 4 * g]);
      const f32x4 w1 = *reinterpret_cast<const f32x4*>(&lds_w[32 * ts + 16 + 4 * g]);
      u32x4 xw[PW];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float lo = 0.f, hi = 0.f;
#pragma unroll
        for (int p = PI - 1; p >= 0; --p) {
          lo += __uint_as_float(xr[p][i] << 16);
          hi += __uint_as_float(xr[p][i] & 0xFFFF0000u);
        }
        lo *= i < 2 ? w0[2 * i] : w1[2 * i - 4];
        hi *= i < 2 ? w0[2 * i + 1] : w1[2 * i - 3];
        uint32_t p3[PW];
        split_pair<PW>(lo, hi, p3);
#pragma unroll
        for (int q = 0; q < PW; ++q) xw[q][i] = p3[q];
      }
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int p = 0; p < PI; ++p) {
          const u32x4 bf = read_tr8(&lds_b[p][0][0], SK, 32 * ts, 16 * kt, lane);
#pragma unroll
          for (int q = 0; q < PW; ++q)
            if (p + q < 3) S[kt] = mfma(bf, xw[q], S[kt]);
        }
    }
    if (bad && lds_first[par][16 * wave + n16] < kL) {
#pragma unroll
      for (int kt = 0; kt < KT; ++kt)
#pragma unroll
        for (int r = 0; r < 4; ++r) S[kt][r] = __builtin_nanf("");
    }
    __syncthreads();   // the chunk's LDS has been read
  }

  // ---- the state after the segment
  if constexpr (STATES) {
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) ws[(size_t)seg * slot + kt * kThreads] = S[kt];
    if (tid == 0 && vb == 0) wd[seg] = (float)total;
  } else if (seg == (used > 0 ? used - 1 : 0)) {
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

template <bool STATES>
ScanFn pick_scan(bool bf16, int dkp) {
  if (bf16) {
    switch (dkp) {
      case 64: return scan_kernel<Bf16, 64, 1, 1, STATES>;
      case 128: return scan_kernel<Bf16, 128, 1, 1, STATES>;
      default: return scan_kernel<Bf16, 256, 1, 1, STATES>;
    }
  }
  return dkp == 64 ? scan_kernel<float, 64, 3, 3, STATES> : scan_kernel<float, 128, 3, 3, STATES>;
}

struct ScanPlan {
  int dkp, vblocks, segs, seg_chunks;
  int64_t blocks;
  size_t state_bytes, bytes;
};

// Sequences are cut into segments that run side by side when heads and
// sequences alone do not fill the chip: about kTarget workgroups (two for each
// of 256 compute units) of equal length. Every segment but a sequence's last is
// read twice (its state first), so one segment is kept where that fills it.
constexpr int64_t kTarget = 512, kMinChunks = 4;

rsq_status plan_scan(const rsq_ssm* p, ScanPlan& w) {
  w.dkp = p->d_k <= 64 ? 64 : p->d_k <= 128 ? 128 : 256;
  w.vblocks = (int)ceil_div(p->d_v, kV);
  const int64_t base = (int64_t)p->heads * w.vblocks;
  const int64_t longest = ceil_div(p->max_len, kL);
  int64_t total = ceil_div(p->tokens, kL) + p->seqs;
  if (total > longest * p->seqs) total = longest * p->seqs;
  int64_t per = ceil_div(total * base, kTarget);
  if (per < kMinChunks) per = kMinChunks;
  if (per > longest) per = longest > 0 ? longest : 1;
  w.segs = (int)(longest > 0 ? ceil_div(longest, per) : 1);
  w.seg_chunks = (int)per;
  w.blocks = base * p->seqs * w.segs;
  if (w.blocks > kMaxGrid) return fail(RSQ_E_UNSUPPORTED, "%lld workgroups", (long long)w.blocks);
  w.state_bytes = w.bytes = 0;
  if (w.segs > 1) {
    w.state_bytes = (size_t)w.blocks * (w.dkp / 16) * kThreads * 16;
    w.bytes = w.state_bytes + (size_t)p->seqs * p->heads * w.segs * 4;
  }
  return RSQ_OK;
}

}  // namespace
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
  if (const rsq_status s = check_ssm_memory(p)) return s;
  ScanPlan w;
  if (const rsq_status s = plan_scan(p, w)) return s;
  if (w.bytes) {
    if (!p->workspace || !aligned(p->workspace, 16)) return fail(RSQ_E_INVALID, "workspace is NULL or not 16-byte aligned");
    if (p->workspace_bytes < w.bytes)
      return fail(RSQ_E_BUFFER, "workspace has %zu bytes, the scan needs %zu", p->workspace_bytes, w.bytes);
  }
  ScanArgs a{};
  a.s = ssm_args(p);
  a.ws_state = static_cast<float*>(p->workspace);
  a.ws_decay = reinterpret_cast<float*>(static_cast<uint8_t*>(p->workspace) + w.state_bytes);
  a.vblocks = w.vblocks, a.segs = w.segs, a.seg_chunks = w.seg_chunks;
  const bool bf16 = p->dtype == RSQ_BF16;
  if (w.segs > 1) {
    hipLaunchKernelGGL(pick_scan<true>(bf16, w.dkp), dim3((unsigned)w.blocks), dim3(kThreads), 0, (hipStream_t)stream, a);
    if (const rsq_status s = launched("selective scan, segment states")) return s;
  }
  hipLaunchKernelGGL(pick_scan<false>(bf16, w.dkp), dim3((unsigned)w.blocks), dim3(kThreads), 0, (hipStream_t)stream, a);
  return launched("selective scan");
}

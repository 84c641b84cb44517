// Attention with a decay for each head (linear.hpp): the C entry points, and the
// single-token form on a dense fp32 state.
#include "linear.hpp"
#include "ssm.hpp"

namespace rsq {
namespace {

constexpr int64_t kMaxRowBytes = 1 << 24;   // rows of the chunked kernels are reached by 32-bit offsets

rsq_status check_linear(const rsq_linear_attn* p, bool prompt) {
  if (!p) return fail(RSQ_E_INVALID, "attn is NULL");
  if (p->dtype != RSQ_F32 && p->dtype != RSQ_BF16) return fail(RSQ_E_INVALID, "dtype %d", p->dtype);
  if (p->seqs < 1 || p->heads < 1) return fail(RSQ_E_INVALID, "seqs %d heads %d", p->seqs, p->heads);
  if (p->key_heads < 1 || p->heads % p->key_heads)
    return fail(RSQ_E_INVALID, "key_heads %d must divide heads %d", p->key_heads, p->heads);
  if (p->d_k < 8 || p->d_v < 8 || p->d_k % 8 || p->d_v % 8)
    return fail(RSQ_E_INVALID, "d_k %d d_v %d must be positive multiples of 8", p->d_k, p->d_v);
  if (p->tokens < 0 || p->tokens > 0x7fffffff) return fail(RSQ_E_INVALID, "tokens %lld", (long long)p->tokens);
  if (p->max_len < 0 || p->max_len > p->tokens)
    return fail(RSQ_E_INVALID, "max_len %lld of %lld tokens", (long long)p->max_len, (long long)p->tokens);
  if (!p->offsets && p->tokens != p->max_len * p->seqs)
    return fail(RSQ_E_INVALID, "without offsets every sequence has max_len rows: %lld tokens, %d of %lld",
                (long long)p->tokens, p->seqs, (long long)p->max_len);
  if (p->d_v > 4096) return fail(RSQ_E_UNSUPPORTED, "d_v %d > 4096", p->d_v);
  const int most = prompt && p->dtype == RSQ_F32 ? 128 : 256;
  if (p->d_k > most) return fail(RSQ_E_UNSUPPORTED, "d_k up to %d with this dtype, got %d", most, p->d_k);
  if (!prompt && (p->offsets || p->max_len != 1)) return fail(RSQ_E_INVALID, "a step takes one row per sequence and no offsets");
  const int64_t vec = p->dtype == RSQ_BF16 ? 8 : 4;
  const int64_t hv = (int64_t)p->heads * p->d_v, hk = (int64_t)p->key_heads * p->d_k;
  if (p->v_stride < hv || p->o_stride < hv || p->q_stride < hk || p->k_stride < hk ||
      (p->alpha && p->alpha_stride != 0 && p->alpha_stride < p->heads) || (p->beta && p->beta_stride < p->heads))
    return fail(RSQ_E_INVALID, "a row stride is shorter than its row");
  if (p->v_stride % vec || p->o_stride % vec || p->q_stride % vec || p->k_stride % vec)
    return fail(RSQ_E_INVALID, "the row strides of q, k, v and o must be multiples of 16 bytes");
  if (prompt) {
    // (the kernels count rows in int, some chunks ahead of the last)
    if (p->max_len > 0x7fffffff - 4096) return fail(RSQ_E_UNSUPPORTED, "max_len %lld", (long long)p->max_len);
    const int64_t size = 16 / vec;
    const int64_t bytes[] = {p->q_stride * size, p->k_stride * size, p->v_stride * size, p->o_stride * size};
    const int64_t strides[] = {p->q_stride, p->k_stride, p->v_stride, p->o_stride};
    for (int i = 0; i < 4; ++i)
      if (strides[i] > kMaxRowBytes || bytes[i] > kMaxRowBytes)
        return fail(RSQ_E_UNSUPPORTED, "rows %lld elements apart, more than 2^24 bytes", (long long)strides[i]);
    if ((p->alpha && p->alpha_stride > kMaxRowBytes / 4) || (p->beta && p->beta_stride > kMaxRowBytes / 4))
      return fail(RSQ_E_UNSUPPORTED, "rows of alpha or beta more than 2^24 bytes apart");
  }
  return RSQ_OK;
}

rsq_status check_linear_memory(const rsq_linear_attn* p) {
  const int size = p->dtype == RSQ_BF16 ? 2 : 4;
  if (p->tokens > 0 && (!p->q || !p->k || !p->v || !p->o)) return fail(RSQ_E_INVALID, "q, k, v and o must be non-NULL");
  if (!p->state) return fail(RSQ_E_INVALID, "state is NULL");
  if (!aligned(p->q, 16) || !aligned(p->k, 16) || !aligned(p->v, 16) || !aligned(p->o, 16) || !aligned(p->state, 16))
    return fail(RSQ_E_INVALID, "q, k, v, o and state must be 16-byte aligned");
  if (!aligned(p->alpha, 4) || !aligned(p->beta, 4) || !aligned(p->offsets, 4))
    return fail(RSQ_E_INVALID, "a pointer is not aligned to its element type");
  const int64_t n = p->tokens, hv = (int64_t)p->heads * p->d_v, hk = (int64_t)p->key_heads * p->d_k;
  const Span written[] = {{p->o, span_bytes(n, p->o_stride, hv, size), "o"},
                          {p->state, (int64_t)p->seqs * p->d_k * hv * 4, "state"},
                          {p->workspace, (int64_t)p->workspace_bytes, "workspace"}};
  const Span read[] = {{p->q, span_bytes(n, p->q_stride, hk, size), "q"},
                       {p->k, span_bytes(n, p->k_stride, hk, size), "k"},
                       {p->v, span_bytes(n, p->v_stride, hv, size), "v"},
                       {p->alpha, p->alpha_stride ? span_bytes(n, p->alpha_stride, p->heads, 4) : (int64_t)p->heads * 4, "alpha"},
                       {p->beta, span_bytes(n, p->beta_stride, p->heads, 4), "beta"},
                       {p->offsets, ((int64_t)p->seqs + 1) * 4, "offsets"}};
  return check_overlap(written, read);
}

LinearArgs linear_args(const rsq_linear_attn* p) {
  LinearArgs a{};
  a.q = p->q, a.k = p->k, a.v = p->v, a.alpha = p->alpha, a.beta = p->beta;
  a.state = p->state, a.o = p->o;
  a.q_stride = p->q_stride, a.k_stride = p->k_stride, a.v_stride = p->v_stride, a.o_stride = p->o_stride;
  a.alpha_stride = p->alpha ? p->alpha_stride : 0, a.beta_stride = p->beta_stride;
  a.s = Sequences{p->offsets, p->tokens, p->max_len, p->seqs};
  a.H = p->heads, a.per_key = p->heads / p->key_heads;
  a.dk = p->d_k, a.dv = p->d_v;
  a.state_in = p->state_in ? 1 : 0;
  return a;
}

// Without write strengths the recurrence is the selective scan's with the decays
// given: x is v, B is k and C is q.
rsq_ssm as_scan(const rsq_linear_attn* p) {
  rsq_ssm s{};
  s.dtype = p->dtype, s.seqs = p->seqs, s.heads = p->heads, s.groups = p->key_heads, s.d_k = p->d_k, s.d_v = p->d_v;
  s.state_in = p->state_in, s.tokens = p->tokens, s.max_len = p->max_len, s.offsets = p->offsets;
  s.x = p->v, s.x_stride = p->v_stride, s.B = p->k, s.b_stride = p->k_stride, s.C = p->q, s.c_stride = p->q_stride;
  s.state = p->state, s.y = p->o, s.y_stride = p->o_stride;
  s.workspace = p->workspace, s.workspace_bytes = p->workspace_bytes;
  return s;
}

// A state of 16 MB and more, which is read and written once, is kept out of the caches: a model
// has one for each layer, and none is still there when its next token comes. Four to 32 states in
// turn, us so and through the caches: 32 heads of 128 x 128 of 64 sequences (134 MB) 51.5, 63, of 32
// 25, 33, of 16 12.9, 17, of 8 9.5, 11.8; of 4 8.1, 7.3. One state alone, which stays in the
// last-level cache, loses by it: of 64 51.5, 47.
constexpr int64_t kPassing = 16 << 20;

// (PASSES is a template's: of a branch between the two the compiler makes one plain access)
typedef float State4 __attribute__((ext_vector_type(4)));
template <bool PASSES>
__device__ __forceinline__ float4 load_state(const float* p) {
  const State4* const at = reinterpret_cast<const State4*>(p);
  State4 v;
  if constexpr (PASSES) v = __builtin_nontemporal_load(at);
  else v = *at;
  return make_float4(v[0], v[1], v[2], v[3]);
}
template <bool PASSES>
__device__ __forceinline__ void store_state(float* p, const float4& m) {
  State4* const at = reinterpret_cast<State4*>(p);
  const State4 v = {m.x, m.y, m.z, m.w};
  if constexpr (PASSES) __builtin_nontemporal_store(v, at);
  else *at = v;
}

// One token: the state is read and written once (8 d_k d_v bytes a head) against 7
// operations an element: bound by memory. With u the token's value,
//   o = a S^T q + (k . q) u,   u = b (v - a S^T k),
// so both sums over the rows come from one reading of the state, which stays in
// registers until u is known. A workgroup owns 64 columns of a head's state (128 take 55 us
// where 64 take 51.5); a thread owns four consecutive columns and every 16th row. The sums meet
// in a fixed order. 64 sequences of 32 heads of 128 x 128 (271 MB) take 51.5 us, 5.3 TB/s, where a
// large copy has 5.1; one sequence 5.1 us, of which an empty launch is 4.6.
constexpr int kColumns = 64, kRows = 16;   // of a workgroup, rows at once

template <typename T, int NR, bool PASSES>
__global__ __launch_bounds__(kColumns / 4 * kRows) void linear_step_kernel(LinearArgs a, int32_t vblocks) {
  constexpr int FOURS = kColumns / 4, WAVES = FOURS * kRows / 64;
  __shared__ float part[WAVES][2][kColumns], part_qk[WAVES];
  const int64_t id = blockIdx.x / vblocks;
  const int vb = blockIdx.x % vblocks;
  const int h = (int)(id % a.H);
  const int64_t s = id / a.H;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int c = threadIdx.x % FOURS, r0 = threadIdx.x / FOURS;
  const int col = vb * kColumns + 4 * c;
  const bool in = col < a.dv;   // (d_v is a multiple of 4)
  const T* q = reinterpret_cast<const T*>(a.q) + s * a.q_stride + (int64_t)(h / a.per_key) * a.dk;
  const T* k = reinterpret_cast<const T*>(a.k) + s * a.k_stride + (int64_t)(h / a.per_key) * a.dk;
  const T* v = reinterpret_cast<const T*>(a.v) + s * a.v_stride + (int64_t)h * a.dv + col;
  float* S = a.state + (size_t)id * a.dk * a.dv + col;
  float4 m[NR];
  float kf[NR], qf[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int row = r0 + i * kRows;
    m[i] = row < a.dk && in && a.state_in ? load_state<PASSES>(S + (size_t)row * a.dv) : make_float4(0.f, 0.f, 0.f, 0.f);
    kf[i] = row < a.dk ? to_f32(k[row]) : 0.f;
    qf[i] = row < a.dk ? to_f32(q[row]) : 0.f;
  }
  const float decay = a.alpha ? a.alpha[s * a.alpha_stride + h] : 1.f;
  const float beta = a.beta ? a.beta[s * a.beta_stride + h] : 0.f;
  float u[4] = {0.f, 0.f, 0.f, 0.f};
  if (in) {
#pragma unroll
    for (int e = 0; e < 4; ++e) u[e] = to_f32(v[e]);
  }
  float ks[4] = {0.f, 0.f, 0.f, 0.f}, qs[4] = {0.f, 0.f, 0.f, 0.f}, qk = 0.f;
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    float* p = &m[i].x;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      p[e] *= decay;
      ks[e] = __builtin_fmaf(kf[i], p[e], ks[e]);
      qs[e] = __builtin_fmaf(qf[i], p[e], qs[e]);
    }
    qk = __builtin_fmaf(kf[i], qf[i], qk);
  }
#pragma unroll
  for (int x = FOURS; x <= 32; x <<= 1) {
#pragma unroll
    for (int e = 0; e < 4; ++e) ks[e] += __shfl_xor(ks[e], x, 64), qs[e] += __shfl_xor(qs[e], x, 64);
    qk += __shfl_xor(qk, x, 64);
  }
  if (lane < FOURS) {
#pragma unroll
    for (int e = 0; e < 4; ++e) part[wave][0][4 * c + e] = ks[e], part[wave][1][4 * c + e] = qs[e];
    if (lane == 0) part_qk[wave] = qk;
  }
  __syncthreads();
  qk = part_qk[0];
#pragma unroll
  for (int w = 1; w < WAVES; ++w) qk += part_qk[w];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int j = 4 * c + e;
    ks[e] = part[0][0][j], qs[e] = part[0][1][j];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) ks[e] += part[w][0][j], qs[e] += part[w][1][j];
    if (a.beta) u[e] = beta * (u[e] - ks[e]);
  }
  if (!in) return;
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int row = r0 + i * kRows;
    if (row < a.dk) {
      float* p = &m[i].x;
#pragma unroll
      for (int e = 0; e < 4; ++e) p[e] = __builtin_fmaf(kf[i], u[e], p[e]);
      store_state<PASSES>(S + (size_t)row * a.dv, m[i]);
    }
  }
  if (r0 == 0) {
    T* o = reinterpret_cast<T*>(a.o) + s * a.o_stride + (int64_t)h * a.dv + col;
#pragma unroll
    for (int e = 0; e < 4; ++e) from_f32(__builtin_fmaf(qk, u[e], qs[e]), o[e]);
  }
}

typedef void (*LinearStepFn)(LinearArgs, int32_t);
template <typename T, bool PASSES>
LinearStepFn pick_step(int dk) {
  return dk <= 64 ? linear_step_kernel<T, 4, PASSES> : dk <= 128 ? linear_step_kernel<T, 8, PASSES> : linear_step_kernel<T, 16, PASSES>;
}

}  // namespace
}  // namespace rsq

using namespace rsq;

extern "C" rsq_status rsq_linear_attention_workspace(const rsq_linear_attn* p, size_t* bytes) {
  if (!bytes) return fail(RSQ_E_INVALID, "bytes is NULL");
  if (const rsq_status s = check_linear(p, true)) return s;
  if (p->beta) return delta_workspace(p, bytes);
  const rsq_ssm scan = as_scan(p);
  return decayed_scan_workspace(&scan, bytes);
}

extern "C" rsq_status rsq_linear_attention(const rsq_linear_attn* p, void* stream) {
  if (const rsq_status s = check_linear(p, true)) return s;
  if (const rsq_status s = check_linear_memory(p)) return s;
  if (p->beta) return run_delta(p, linear_args(p), stream);
  const rsq_ssm scan = as_scan(p);
  return run_decayed_scan(&scan, p->alpha, p->alpha_stride, stream);
}

extern "C" rsq_status rsq_linear_attention_step(const rsq_linear_attn* p, void* stream) {
  if (const rsq_status s = check_linear(p, false)) return s;
  if (const rsq_status s = check_linear_memory(p)) return s;
  constexpr int threads = kColumns / 4 * kRows;
  const int64_t vblocks = ceil_div(p->d_v, kColumns);
  const int64_t blocks = (int64_t)p->seqs * p->heads * vblocks;
  if (const rsq_status s = check_blocks(blocks, threads)) return s;
  const bool passes = (int64_t)p->seqs * p->heads * p->d_k * p->d_v * 4 >= kPassing;
  const LinearStepFn fn = p->dtype == RSQ_BF16 ? (passes ? pick_step<Bf16, true> : pick_step<Bf16, false>)(p->d_k)
                                               : (passes ? pick_step<float, true> : pick_step<float, false>)(p->d_k);
  hipLaunchKernelGGL(fn, dim3((unsigned)blocks), dim3(threads), 0, (hipStream_t)stream, linear_args(p), (int32_t)vblocks);
  return launched("linear attention step");
}

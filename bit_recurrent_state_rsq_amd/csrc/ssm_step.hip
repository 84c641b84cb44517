// One token of the selective state-space recurrence (ssm.hpp) for every
// sequence, on a dense fp32 state updated in place, and the argument checks
// that it shares with the prompt scan.
#include "ssm.hpp"

namespace rsq {

rsq_status check_ssm(const rsq_ssm* p, bool prompt) {
  if (!p) return fail(RSQ_E_INVALID, "ssm is NULL");
  if (p->dtype != RSQ_F32 && p->dtype != RSQ_BF16) return fail(RSQ_E_INVALID, "dtype %d", p->dtype);
  if (p->seqs < 1 || p->heads < 1) return fail(RSQ_E_INVALID, "seqs %d heads %d", p->seqs, p->heads);
  if (p->groups < 1 || p->heads % p->groups)
    return fail(RSQ_E_INVALID, "groups %d must divide heads %d", p->groups, p->heads);
  if (p->d_k < 8 || p->d_v < 8 || p->d_k % 8 || p->d_v % 8)
    return fail(RSQ_E_INVALID, "d_k %d d_v %d must be positive multiples of 8", p->d_k, p->d_v);
  if (p->tokens < 0 || p->tokens > 0x7fffffff) return fail(RSQ_E_INVALID, "tokens %lld", (long long)p->tokens);
  if (p->max_len < 0 || p->max_len > p->tokens)
    return fail(RSQ_E_INVALID, "max_len %lld of %lld tokens", (long long)p->max_len, (long long)p->tokens);
  if (!p->offsets && p->tokens != p->max_len * p->seqs)
    return fail(RSQ_E_INVALID, "without offsets every sequence has max_len rows: %lld tokens, %d of %lld",
                (long long)p->tokens, p->seqs, (long long)p->max_len);
  if (prompt) {
    if (p->d_v > 4096) return fail(RSQ_E_UNSUPPORTED, "d_v %d > 4096", p->d_v);
    const int most = p->dtype == RSQ_BF16 ? 256 : 128;
    if (p->d_k > most)
      return fail(RSQ_E_UNSUPPORTED, "the scan takes d_k up to %d with this dtype, got %d", most, p->d_k);
  } else {
    if (p->offsets || p->max_len != 1) return fail(RSQ_E_INVALID, "a step takes one row per sequence and no offsets");
    if (p->d_v > 1024) return fail(RSQ_E_UNSUPPORTED, "d_v %d > 1024", p->d_v);
    if (p->d_k > 4096) return fail(RSQ_E_UNSUPPORTED, "d_k %d > 4096", p->d_k);
  }
  const int64_t vec = p->dtype == RSQ_BF16 ? 8 : 4;
  const int64_t hv = (int64_t)p->heads * p->d_v, gk = (int64_t)p->groups * p->d_k;
  if (p->x_stride < hv || p->y_stride < hv || p->b_stride < gk || p->c_stride < gk || p->dt_stride < p->heads)
    return fail(RSQ_E_INVALID, "a row stride is shorter than its row");
  if (p->x_stride % vec || p->y_stride % vec || p->b_stride % vec || p->c_stride % vec)
    return fail(RSQ_E_INVALID, "the row strides of x, B, C and y must be multiples of 16 bytes");
  return RSQ_OK;
}

namespace {

// the memory that a call writes and reads, but for its state
int64_t ssm_span(const rsq_ssm* p, int64_t stride, int64_t cols) {
  return span_bytes(p->tokens, stride, cols, p->dtype == RSQ_BF16 ? 2 : 4);
}
Span y_span(const rsq_ssm* p) { return {p->y, ssm_span(p, p->y_stride, (int64_t)p->heads * p->d_v), "y"}; }
Span work_span(const rsq_ssm* p) { return {p->workspace, (int64_t)p->workspace_bytes, "workspace"}; }
struct ReadSpans {
  Span s[8];
};
ReadSpans read_spans(const rsq_ssm* p) {
  const int64_t gk = (int64_t)p->groups * p->d_k, hb = (int64_t)p->heads * 4;
  return {{{p->x, ssm_span(p, p->x_stride, (int64_t)p->heads * p->d_v), "x"},
           {p->B, ssm_span(p, p->b_stride, gk), "B"},
           {p->C, ssm_span(p, p->c_stride, gk), "C"},
           {p->dt, ssm_span(p, p->dt_stride, p->heads), "dt"},
           {p->A, hb, "A"},
           {p->D, hb, "D"},
           {p->dt_bias, hb, "dt_bias"},
           {p->offsets, ((int64_t)p->seqs + 1) * 4, "offsets"}}};
}

}  // namespace

rsq_status check_ssm_memory(const rsq_ssm* p) {
  const int size = p->dtype == RSQ_BF16 ? 2 : 4;
  if (p->tokens > 0 && (!p->x || !p->B || !p->C || !p->dt || !p->y))
    return fail(RSQ_E_INVALID, "x, B, C, dt and y must be non-NULL");
  if (!p->A) return fail(RSQ_E_INVALID, "A is NULL");
  if (!aligned(p->x, 16) || !aligned(p->B, 16) || !aligned(p->C, 16) || !aligned(p->y, 16) || !aligned(p->state, 16))
    return fail(RSQ_E_INVALID, "x, B, C, y and state must be 16-byte aligned");
  if (!aligned(p->dt, size) || !aligned(p->A, 4) || !aligned(p->D, 4) || !aligned(p->dt_bias, 4) ||
      !aligned(p->offsets, 4))
    return fail(RSQ_E_INVALID, "a pointer is not aligned to its element type");
  const Span written[] = {y_span(p), {p->state, (int64_t)p->seqs * p->d_k * p->heads * p->d_v * 4, "state"}, work_span(p)};
  return check_overlap(written, read_spans(p).s);
}

rsq_status check_ssm_apart(const rsq_ssm* p, const Span& range) {
  const Span written[] = {range, y_span(p), work_span(p)};
  return check_overlap(written, read_spans(p).s);
}

SsmArgs ssm_args(const rsq_ssm* p) {
  SsmArgs a{};
  a.x = p->x, a.B = p->B, a.C = p->C, a.dt = p->dt, a.A = p->A, a.D = p->D, a.dt_bias = p->dt_bias;
  a.state = p->state, a.y = p->y;
  a.x_stride = p->x_stride, a.b_stride = p->b_stride, a.c_stride = p->c_stride;
  a.dt_stride = p->dt_stride, a.y_stride = p->y_stride;
  a.q = Sequences{p->offsets, p->tokens, p->max_len, p->seqs};
  a.H = p->heads, a.per_group = p->heads / p->groups;
  a.dk = p->d_k, a.dv = p->d_v;
  a.softplus = p->softplus ? 1 : 0, a.state_in = p->state_in ? 1 : 0;
  return a;
}

namespace {

// The state is read and written once (8 d_k d_v bytes a head) against 5
// operations an element: bound by memory. A workgroup owns one head's state; a
// thread owns four consecutive columns, so that rows are read in whole, and
// every rows-th run of rows, kAhead of them in flight. The sums over the rows
// meet in LDS in a fixed order. 128 sequences of 64 heads of 128 x 64 (539 MB) take
// 106 us, 5.1 TB/s (a large copy moves 4.9); one sequence 5.3 us, where an empty
// launch takes 4.6.
constexpr int kAhead = 8;

template <typename T>
__global__ __launch_bounds__(256) void ssm_step_kernel(SsmArgs a) {
  extern __shared__ float part[];   // [rows at once][dv]
  const int h = blockIdx.x % a.H;
  const int64_t s = blockIdx.x / a.H;
  const int cols = a.dv / 4;                 // column fours, <= 256
  const int rows = 256 / cols;               // rows at once
  const int c = threadIdx.x % cols, r0 = threadIdx.x / cols;
  const int group = h / a.per_group;
  const float d = ssm_delta<T>(a, s, h);
  const float decay = expf(d * a.A[h]);
  const T* x = reinterpret_cast<const T*>(a.x) + s * a.x_stride + (int64_t)h * a.dv;
  const T* B = reinterpret_cast<const T*>(a.B) + s * a.b_stride + (int64_t)group * a.dk;
  const T* C = reinterpret_cast<const T*>(a.C) + s * a.c_stride + (int64_t)group * a.dk;
  float4* S = reinterpret_cast<float4*>(a.state + ((size_t)s * a.H + h) * a.dk * a.dv) + c;
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  if (r0 < rows) {
    float dx[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) dx[e] = d * to_f32(x[4 * c + e]);
    for (int k0 = r0; k0 < a.dk; k0 += rows * kAhead) {
      float4 v[kAhead];
      float b[kAhead], q[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int k = k0 + i * rows;
        if (k < a.dk) {
          v[i] = a.state_in ? S[(size_t)k * cols] : make_float4(0.f, 0.f, 0.f, 0.f);
          b[i] = to_f32(B[k]), q[i] = to_f32(C[k]);
        }
      }
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const int k = k0 + i * rows;
        if (k < a.dk) {
          float* p = &v[i].x;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            p[e] = __builtin_fmaf(b[i], dx[e], decay * p[e]);
            acc[e] = __builtin_fmaf(q[i], p[e], acc[e]);
          }
          S[(size_t)k * cols] = v[i];
        }
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) part[r0 * a.dv + 4 * c + e] = acc[e];
  }
  __syncthreads();
  T* y = reinterpret_cast<T*>(a.y) + s * a.y_stride + (int64_t)h * a.dv;
  const float Dh = a.D ? a.D[h] : 0.f;
  for (int j = threadIdx.x; j < a.dv; j += 256) {
    float o = part[j];
    for (int r = 1; r < rows; ++r) o += part[r * a.dv + j];
    if (a.D) o = __builtin_fmaf(Dh, to_f32(x[j]), o);
    from_f32(o, y[j]);
  }
}

// Inputs of a decode step on a quantized state: a workgroup per head and
// sequence. They are d_k + d_v elements a head against the d_k d_v of the state
// that the step then moves: two launches more (these and the skip connection),
// 41 us against 30 for the step alone (128 sequences, 64 heads of 128 x 64, INT8).
template <typename T>
__global__ __launch_bounds__(128) void ssm_gates_kernel(SsmArgs a, SsmGates o) {
  const int64_t tile = blockIdx.x;
  const int h = (int)(tile % a.H);
  const int64_t s = tile / a.H;
  const int group = h / a.per_group;
  const float d = ssm_delta<T>(a, s, h);
  if (threadIdx.x == 0) o.alpha[tile] = expf(d * a.A[h]);
  const T* x = reinterpret_cast<const T*>(a.x) + s * a.x_stride + (int64_t)h * a.dv;
  const T* B = reinterpret_cast<const T*>(a.B) + s * a.b_stride + (int64_t)group * a.dk;
  const T* C = reinterpret_cast<const T*>(a.C) + s * a.c_stride + (int64_t)group * a.dk;
  for (int i = threadIdx.x; i < a.dk; i += 128) {
    reinterpret_cast<T*>(o.q)[tile * a.dk + i] = C[i];
    reinterpret_cast<T*>(o.k)[tile * a.dk + i] = B[i];
  }
  for (int j = threadIdx.x; j < a.dv; j += 128) from_f32(d * to_f32(x[j]), reinterpret_cast<T*>(o.v)[tile * a.dv + j]);
}

template <typename T>
__global__ __launch_bounds__(256) void ssm_skip_kernel(SsmArgs a, const float* o) {
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t hv = (int64_t)a.H * a.dv;
  const int64_t s = id / hv;
  if (s >= a.q.seqs) return;
  const int64_t j = id - s * hv;
  float y = o[id];
  if (a.D) y = __builtin_fmaf(a.D[j / a.dv], to_f32(reinterpret_cast<const T*>(a.x)[s * a.x_stride + j]), y);
  from_f32(y, reinterpret_cast<T*>(a.y)[s * a.y_stride + j]);
}

}  // namespace

rsq_status check_ssm_launches(const SsmArgs& a) {
  if (const rsq_status s = check_blocks((int64_t)a.q.seqs * a.H, 128)) return s;
  return check_blocks(ceil_div((int64_t)a.q.seqs * a.H * a.dv, 256), 256);
}

rsq_status launch_ssm_gates(const SsmArgs& a, bool bf16, const SsmGates& out, void* stream) {
  const unsigned tiles = (unsigned)((int64_t)a.q.seqs * a.H);
  if (bf16) hipLaunchKernelGGL(ssm_gates_kernel<Bf16>, dim3(tiles), dim3(128), 0, (hipStream_t)stream, a, out);
  else hipLaunchKernelGGL(ssm_gates_kernel<float>, dim3(tiles), dim3(128), 0, (hipStream_t)stream, a, out);
  return launched("step gates");
}

rsq_status launch_ssm_skip(const SsmArgs& a, bool bf16, const float* o, void* stream) {
  const unsigned blocks = (unsigned)ceil_div((int64_t)a.q.seqs * a.H * a.dv, 256);
  if (bf16) hipLaunchKernelGGL(ssm_skip_kernel<Bf16>, dim3(blocks), dim3(256), 0, (hipStream_t)stream, a, o);
  else hipLaunchKernelGGL(ssm_skip_kernel<float>, dim3(blocks), dim3(256), 0, (hipStream_t)stream, a, o);
  return launched("step skip connection");
}

}  // namespace rsq

using namespace rsq;

extern "C" rsq_status rsq_ssm_step(const rsq_ssm* p, void* stream) {
  if (const rsq_status s = check_ssm(p, false)) return s;
  if (!p->state) return fail(RSQ_E_INVALID, "state is NULL");
  if (const rsq_status s = check_ssm_memory(p)) return s;
  const int64_t blocks = (int64_t)p->seqs * p->heads;
  if (const rsq_status s = check_blocks(blocks, 256)) return s;
  const SsmArgs a = ssm_args(p);
  const size_t lds = (size_t)(256 / (p->d_v / 4)) * p->d_v * sizeof(float);   // at most 4 KB
  if (p->dtype == RSQ_BF16)
    hipLaunchKernelGGL(ssm_step_kernel<Bf16>, dim3((unsigned)blocks), dim3(256), lds, (hipStream_t)stream, a);
  else
    hipLaunchKernelGGL(ssm_step_kernel<float>, dim3((unsigned)blocks), dim3(256), lds, (hipStream_t)stream, a);
  return launched("selective scan step");
}

// Arguments and gates of the selective state-space recurrence
//   d = softplus(dt + dt_bias) (or dt + dt_bias),  a = exp(d A),
//   S_t = a S_{t-1} + d B_t x_t^T,   y_t = S_t^T C_t + D x_t,
// shared by the prompt scan and its single-token forms. Heads h of a group
// g = h / (heads / groups) share B and C.
#pragma once
#include "layer_ops.hpp"

namespace rsq {

struct SsmArgs {
  const void* x;
  const void* B;
  const void* C;
  const void* dt;
  const float* A;
  const float* D;
  const float* dt_bias;
  float* state;
  void* y;
  int64_t x_stride, b_stride, c_stride, dt_stride, y_stride;
  Sequences q;
  int32_t H, per_group;   // heads, heads of a group
  int32_t dk, dv;
  int32_t softplus, state_in;
};

// log(1 + e^z) without overflow: max(z, 0) + log1p(t), t = e^-|z| <= 1, with
// log1p(t) = 2 artanh(q), q = t / (2 + t) <= 1/3, by its series to q^15 (the next
// term is below 2^-28 of the sum): a third of log1pf's instructions, in the scan on the
// path that each chunk waits for. Within 5 x 2^-24 of the value.
__device__ __forceinline__ float softplus(float z) {
  const float t = expf(-fabsf(z)), d = 2.f + t;
  const float r = __builtin_amdgcn_rcpf(d);
  float q = t * r;
  q = __builtin_fmaf(__builtin_fmaf(-q, d, t), r, q);
  const float s = q * q;
  float p = 1.f / 15.f;
  p = __builtin_fmaf(p, s, 1.f / 13.f);
  p = __builtin_fmaf(p, s, 1.f / 11.f);
  p = __builtin_fmaf(p, s, 1.f / 9.f);
  p = __builtin_fmaf(p, s, 1.f / 7.f);
  p = __builtin_fmaf(p, s, 1.f / 5.f);
  p = __builtin_fmaf(p, s, 1.f / 3.f);
  q *= 2.f;
  return fmaxf(z, 0.f) + __builtin_fmaf(q, s * p, q);
}

template <typename T>
__device__ __forceinline__ float ssm_delta(const SsmArgs& a, int64_t row, int h) {
  float z = to_f32(reinterpret_cast<const T*>(a.dt)[row * a.dt_stride + h]);
  if (a.dt_bias) z += a.dt_bias[h];
  return a.softplus ? softplus(z) : z;
}

}  // namespace rsq

// ---------------------------------------------------------------- host side
#include "host_util.hpp"

namespace rsq {

// Shapes, types and strides of a scan (`prompt`) or a single-token step.
rsq_status check_ssm(const rsq_ssm* p, bool prompt);
// Pointers: present, aligned, outputs apart from everything else.
rsq_status check_ssm_memory(const rsq_ssm* p);
// A written range outside the arguments is apart from all of them.
rsq_status check_ssm_apart(const rsq_ssm* p, const Span& written);
SsmArgs ssm_args(const rsq_ssm* p);

// The scan with given decays: S = alpha S + B x^T, y = S^T C (A, dt, dt_bias and D are
// not looked at, the other arguments have been checked). alpha: fp32 [tokens][heads], rows
// alpha_stride apart (0: one row for all tokens), or NULL for 1.
rsq_status decayed_scan_workspace(const rsq_ssm* p, size_t* bytes);
rsq_status run_decayed_scan(const rsq_ssm* p, const float* alpha, int64_t alpha_stride, void* stream);

// The decode step's inputs of one token: q and k from the head's C and B, v =
// delta x rounded to the inputs' type (the decode step takes q, k and v of one
// type; of bf16 inputs that is 2^-8 of what the token adds, where an 8-bit state's
// own codes are steps of 2^-7 of their group's largest), alpha = exp(delta A).
struct SsmGates {
  void* q;
  void* k;
  void* v;
  float* alpha;
};
// Refuses what the two launches below cannot have.
rsq_status check_ssm_launches(const SsmArgs& a);
rsq_status launch_ssm_gates(const SsmArgs& a, bool bf16, const SsmGates& out, void* stream);
// y = o + D x
rsq_status launch_ssm_skip(const SsmArgs& a, bool bf16, const float* o, void* stream);

}  // namespace rsq

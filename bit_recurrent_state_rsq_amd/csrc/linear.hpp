// Attention with a decay for each head, with or without the delta rule:
//   u_t = v_t,  or with write strengths b_t  u_t = b_t (v_t - a_t S_{t-1}^T k_t),
//   S_t = a_t S_{t-1} + k_t u_t^T,   o_t = S_t^T q_t.
// Heads h share the keys and queries of key head h / (heads / key_heads).
#pragma once
#include "host_util.hpp"
#include "layer_ops.hpp"

namespace rsq {

struct LinearArgs {
  const void* q;
  const void* k;
  const void* v;
  const float* alpha;   // NULL: 1
  const float* beta;
  float* state;
  void* o;
  int64_t q_stride, k_stride, v_stride, o_stride, alpha_stride, beta_stride;   // alpha_stride 0: one row for all tokens
  Sequences s;
  int32_t H, per_key;   // heads, heads of a key head
  int32_t dk, dv;
  int32_t state_in;
};

// Prompts with the delta rule; the arguments have been checked.
rsq_status delta_workspace(const rsq_linear_attn* p, size_t* bytes);
rsq_status run_delta(const rsq_linear_attn* p, const LinearArgs& a, void* stream);

}  // namespace rsq

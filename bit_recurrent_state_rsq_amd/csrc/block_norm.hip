// Norms of rows before and after a block, with the block's gate and residual:
//   u = x              (gate_first: x * act(gate))
//   u = u / sqrt(mean(u^2) + eps) * weight, the mean over `group` columns or the row
//   u = u * act(gate)  (unless it came first)
//   h = residual + residual_scale * u, stored back rounded to its type (no residual: h = u)
//   y = h / sqrt(mean(h^2) + eps) * next_weight (without next_weight: h), or its 8-bit codes
// all in fp32 between the loads and the stores; each part may be left out.
//
// Bound by memory: every operand is read once and every result written once, a row
// staying in registers between its sums and its output. Each part as a call of its own
// would write u and h and read them again. 16384 x 2048 bf16 with a residual between
// two norms (268 MB) takes 53 to 55 us, 5 TB/s, as much as a large copy; 16 rows of 4096,
// normed by heads of 128, gated, to E4M3 6.0 us, of which an empty launch is 4.6.
#include <type_traits>

#include "host_util.hpp"
#include "norm.hpp"

namespace rsq {
namespace {

struct BlockArgs {
  const void* x;
  const void* gate;
  void* residual;
  const float* weight;
  const float* next_weight;
  void* y;
  float* scales;
  int64_t x_stride, g_stride, r_stride, y_stride;
  int64_t rows;
  int32_t cols, group, weight_cols, scale_group;   // group, scale_group 0: the row
  int32_t activation, gate_first;
  float eps, residual_scale;
  int32_t wide;   // bits 0 to 5: x, gate, residual, y, weight, next_weight take 16-byte (codes: 8-byte) accesses
};

// e^-v is an infinity for v below about -88, and the quotient then zero: sigmoid is
// below fp32's normal numbers there, and silu's value, 2.4e-37 at most, is given as zero
__device__ __forceinline__ float activate(float v, int act) {
  if (act == RSQ_ACT_NONE) return v;
  return (act == RSQ_ACT_SILU ? v : 1.f) / (1.f + expf(-v));
}

template <int R, int NV>
__device__ __forceinline__ float square_sum(const float (&h)[NV][kCols]) {
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < kCols; ++e) sum = __builtin_fmaf(h[i][e], h[i][e], sum);
  return sum;
}

// R threads a row, up to NV * kCols columns a thread.
template <typename T, int OUT, int R, int NV>
__global__ __launch_bounds__(R < 256 ? 256 : R) void block_norm_kernel(BlockArgs a) {
  constexpr int ROWS = R < 256 ? 256 / R : 1;
  __shared__ uint32_t lds[16];
  __shared__ float part[ROWS][NV * R];   // sums of eight columns, where a group is not 1, 2, 4, ... 64 of them
  const int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / R;
  const int tid = threadIdx.x % R;
  // R < 256: a row belongs to one wavefront, nothing below crosses it
  if (row >= a.rows) return;
  const T* x = reinterpret_cast<const T*>(a.x) + row * a.x_stride;
  const T* gate = a.gate ? reinterpret_cast<const T*>(a.gate) + row * a.g_stride : nullptr;
  T* res = a.residual ? reinterpret_cast<T*>(a.residual) + row * a.r_stride : nullptr;
  // All of a row's inputs are on their way at once; of 32 columns a thread they would not
  // all fit its registers, and gate and residual are read where they are used.
  constexpr bool EARLY = NV <= 2;
  constexpr int NE = EARLY ? NV : 1;
  float h[NV][kCols], g[NE][kCols], r[NE][kCols];
#pragma unroll
  for (int i = 0; i < NV; ++i) load_cols(x, (i * R + tid) * kCols, a.cols, a.wide & 1, h[i]);
  if (EARLY && gate)
#pragma unroll
    for (int i = 0; i < NE; ++i) load_cols(gate, (i * R + tid) * kCols, a.cols, a.wide & 2, g[i]);
  if (EARLY && res)
#pragma unroll
    for (int i = 0; i < NE; ++i) load_cols(res, (i * R + tid) * kCols, a.cols, a.wide & 4, r[i]);
  auto apply_gate = [&]() {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float (&v)[kCols] = g[EARLY ? i : 0];
      if (!EARLY) load_cols(gate, (i * R + tid) * kCols, a.cols, a.wide & 2, v);
#pragma unroll
      for (int e = 0; e < kCols; ++e) h[i][e] *= activate(v[e], a.activation);
    }
  };
  if (gate && a.gate_first) apply_gate();
  if (a.weight) {
    float rstd[NV];
    if (a.group == 0) {
      const float sum = __uint_as_float(row_reduce<R, true>(__float_as_uint(square_sum<R, NV>(h)), lds));
      const float s = 1.f / sqrtf(sum / (float)a.cols + a.eps);
#pragma unroll
      for (int i = 0; i < NV; ++i) rstd[i] = s;
    } else {
      const int lanes = a.group / kCols;   // threads of a group
      float sums[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        sums[i] = 0.f;
#pragma unroll
        for (int e = 0; e < kCols; ++e) sums[i] = __builtin_fmaf(h[i][e], h[i][e], sums[i]);
      }
      if (lanes <= 64 && (lanes & (lanes - 1)) == 0) {
        for (int s = 1; s < lanes; s <<= 1)
#pragma unroll
          for (int i = 0; i < NV; ++i) sums[i] += __shfl_xor(sums[i], s, 64);
      } else {
        // Of any other group a thread adds up the sums of eight columns alone, which large groups
        // pay for: 4096 rows of 16384 bf16 columns in groups of 1024 84 us, of 4096 237, of 16384
        // 909, where groups of up to 512 and whole rows take 58.
        float* const p = part[R < 256 ? threadIdx.x / R : 0];
#pragma unroll
        for (int i = 0; i < NV; ++i) p[i * R + tid] = sums[i];
        if constexpr (R > 64) __syncthreads();
        else __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int first = (i * R + tid) / lanes * lanes;
          sums[i] = 0.f;
          if (first * kCols < a.cols)
            for (int s = 0; s < lanes; ++s) sums[i] += p[first + s];
        }
      }
#pragma unroll
      for (int i = 0; i < NV; ++i)   // (threads without columns stay at zero, with an eps of zero too)
        rstd[i] = (i * R + tid) * kCols < a.cols ? 1.f / sqrtf(sums[i] / (float)a.group + a.eps) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * R + tid) * kCols;
      float w[kCols];
      // (one weight for all groups, of which eight columns are in one; or one for the row)
      if (a.weight_cols == a.cols) load_cols(a.weight, c, a.cols, a.wide & 16, w);
      else load_cols(a.weight, c % a.weight_cols, a.weight_cols, a.wide & 16, w);
#pragma unroll
      for (int e = 0; e < kCols; ++e) h[i][e] = h[i][e] * rstd[i] * w[e];
    }
  }
  if (gate && !a.gate_first) apply_gate();
  if (res)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float (&v)[kCols] = r[EARLY ? i : 0];
      if (!EARLY) load_cols(res, (i * R + tid) * kCols, a.cols, a.wide & 4, v);
#pragma unroll
      for (int e = 0; e < kCols; ++e) h[i][e] = __builtin_fmaf(a.residual_scale, h[i][e], v[e]);
      store_cols(res, (i * R + tid) * kCols, a.cols, a.wide & 4, h[i]);
    }
  if (!a.y) return;
  if (a.next_weight) {
    const float sum = __uint_as_float(row_reduce<R, true>(__float_as_uint(square_sum<R, NV>(h)), lds));
    const float s = 1.f / sqrtf(sum / (float)a.cols + a.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float w[kCols];
      load_cols(a.next_weight, (i * R + tid) * kCols, a.cols, a.wide & 32, w);
#pragma unroll
      for (int e = 0; e < kCols; ++e) h[i][e] = h[i][e] * s * w[e];
    }
  }
  store_row<OUT, R, NV>(h, a.y, a.scales, row, a.y_stride, a.cols, a.scale_group, a.wide & 8, tid, lds);
}

typedef void (*BlockFn)(BlockArgs);
struct BlockPick {
  BlockFn fn;
  int threads, rows;
};

// A wavefront a row up to 1024 columns (its sums need no barrier), then 256, 512 and
// 1024 threads with 8 or 16 columns each; of 32, more is read late (EARLY), which only
// more long rows than there are compute units make up for: two are then on a unit. us of
// bf16 rows with a residual between two norms; of heads normed, gated, to int8, on operands
// past the last-level cache: 16384 rows of 512 columns 18; 20 (16 columns a thread 21; 26),
// 1024 31; 33 (256 threads 41; 49), 2048 53; 60 (a wavefront 59; 61, 512 threads 77; 94),
// 4096 103; 112 (512 threads 103; 116, 1024 156; 193), 8192 204; 218 (256 threads 206; 219,
// 1024 209; 240). 16384 columns, 512 threads against 1024: 4096 rows 112; 126 against 121;
// 152, 512 rows 18; 21 against 20; 23, 257 rows 13; 19 against 17; 21, but 256 rows 12.4;
// 14.9 against 11.3; 12.6. 16 rows of 2048 columns 3.8; 4.5 (a wavefront 5.2; 8.5), of 4096
// 4.3; 6.0 (512 threads 3.9; 5.0), of 8192 4.6; 6.9 (1024 4.3; 6.1).
constexpr int64_t kUnits = 256;   // compute units
template <typename T, int OUT>
BlockPick pick(int cols, int64_t rows) {
  if (cols <= 512) return {block_norm_kernel<T, OUT, 64, 1>, 256, 4};
  if (cols <= 1024) return {block_norm_kernel<T, OUT, 64, 2>, 256, 4};
  if (cols <= 2048) return {block_norm_kernel<T, OUT, 256, 1>, 256, 1};
  if (cols <= 4096) return {block_norm_kernel<T, OUT, 256, 2>, 256, 1};
  if (cols <= 8192) return {block_norm_kernel<T, OUT, 512, 2>, 512, 1};
  if (cols <= 16384 && rows > kUnits) return {block_norm_kernel<T, OUT, 512, 4>, 512, 1};
  if (cols <= 16384) return {block_norm_kernel<T, OUT, 1024, 2>, 1024, 1};
  return {block_norm_kernel<T, OUT, 1024, 4>, 1024, 1};
}

template <typename T>
BlockPick pick_out(int out, int cols, int64_t rows) {
  switch (out) {
    case RSQ_F32: return pick<T, kOutF32>(cols, rows);
    case RSQ_BF16: return pick<T, kOutBf16>(cols, rows);
    case RSQ_INT8: return pick<T, kOutInt8>(cols, rows);
    default: return pick<T, kOutE4m3>(cols, rows);
  }
}

}  // namespace
}  // namespace rsq

using namespace rsq;

extern "C" rsq_status rsq_block_norm(const rsq_block* p, void* stream) {
  if (!p) return fail(RSQ_E_INVALID, "block is NULL");
  if (p->dtype != RSQ_F32 && p->dtype != RSQ_BF16) return fail(RSQ_E_INVALID, "dtype %d", p->dtype);
  const bool codes = p->out_dtype == RSQ_INT8 || p->out_dtype == RSQ_E4M3;
  if (!codes && p->out_dtype != RSQ_F32 && p->out_dtype != RSQ_BF16)
    return fail(RSQ_E_INVALID, "out_dtype %d", p->out_dtype);
  if (p->rows < 0 || p->rows > 0x7fffffff || p->cols < 1)
    return fail(RSQ_E_INVALID, "rows %lld cols %d", (long long)p->rows, p->cols);
  if (p->cols > 32768) return fail(RSQ_E_UNSUPPORTED, "cols %d > 32768", p->cols);
  if (!(p->eps >= 0.f) || p->eps > 3.4e38f) return fail(RSQ_E_INVALID, "eps must be finite and >= 0");
  if (!(p->residual_scale >= -3.4e38f && p->residual_scale <= 3.4e38f)) return fail(RSQ_E_INVALID, "residual_scale must be finite");
  if (p->activation != RSQ_ACT_NONE && p->activation != RSQ_ACT_SILU && p->activation != RSQ_ACT_SIGMOID)
    return fail(RSQ_E_INVALID, "activation %d", p->activation);
  if (p->group < 0 || p->group % 8 || (p->group && p->cols % p->group))
    return fail(RSQ_E_INVALID, "group %d: 0, or a multiple of 8 that divides cols %d", p->group, p->cols);
  if (p->group && !p->weight) return fail(RSQ_E_INVALID, "group goes with weight");
  if (p->weight && p->weight_cols != p->cols && (!p->group || p->weight_cols != p->group))
    return fail(RSQ_E_INVALID, "weight_cols %d: cols %d, or the group %d", p->weight_cols, p->cols, p->group);
  if (p->scale_group != 0 && (!codes || (p->scale_group != 32 && p->scale_group != 64 && p->scale_group != 128) || p->cols % p->scale_group))
    return fail(RSQ_E_INVALID, "scale_group %d: 0, or 32, 64 or 128 dividing cols %d with an 8-bit output", p->scale_group, p->cols);
  if (p->rows == 0) return RSQ_OK;   // (an empty tensor has no address)
  if (!p->x) return fail(RSQ_E_INVALID, "x is NULL");
  if (!p->residual && p->residual_scale != 1.f) return fail(RSQ_E_INVALID, "residual_scale goes with a residual");
  if (!p->y && (!p->residual || p->next_weight || codes))
    return fail(RSQ_E_INVALID, "y may be NULL only where the residual is the result: with it, without next_weight and codes");
  if (codes != (p->scales != nullptr)) return fail(RSQ_E_INVALID, "scales are given with an 8-bit output, and only there");
  if (p->x_stride < p->cols || (p->y && p->y_stride < p->cols) || (p->residual && p->residual_stride < p->cols) ||
      (p->gate && p->gate_stride < p->cols))
    return fail(RSQ_E_INVALID, "a row stride is below %d columns", p->cols);
  const int size = p->dtype == RSQ_BF16 ? 2 : 4;
  const int osize = codes ? 1 : p->out_dtype == RSQ_BF16 ? 2 : 4;
  if (!aligned(p->x, size) || !aligned(p->gate, size) || !aligned(p->residual, size) || !aligned(p->y, osize) ||
      !aligned(p->weight, 4) || !aligned(p->next_weight, 4) || !aligned(p->scales, 4))
    return fail(RSQ_E_INVALID, "a pointer is not aligned to its element type");
  const int64_t nscales = p->rows * (p->scale_group ? p->cols / p->scale_group : 1);
  const Span written[] = {{p->y, span_bytes(p->rows, p->y_stride, p->cols, osize), "y"},
                          {p->residual, span_bytes(p->rows, p->residual_stride, p->cols, size), "residual"},
                          {p->scales, nscales * 4, "scales"}};
  const Span read[] = {{p->x, span_bytes(p->rows, p->x_stride, p->cols, size), "x"},
                       {p->gate, span_bytes(p->rows, p->gate_stride, p->cols, size), "gate"},
                       {p->weight, (int64_t)p->weight_cols * 4, "weight"},
                       {p->next_weight, (int64_t)p->cols * 4, "next_weight"}};
  if (const rsq_status s = check_overlap(written, read)) return s;

  BlockArgs a{};
  a.weight = p->weight, a.next_weight = p->next_weight;
  a.x_stride = p->x_stride, a.g_stride = p->gate_stride, a.r_stride = p->residual_stride, a.y_stride = p->y_stride;
  a.cols = p->cols, a.group = p->group, a.weight_cols = p->weight_cols, a.scale_group = p->scale_group;
  a.activation = p->activation, a.gate_first = p->gate_first ? 1 : 0;
  a.eps = p->eps, a.residual_scale = p->residual_scale;
  auto wide = [](const void* q, int64_t stride, int sz, int n) { return q && aligned(q, n) && stride * sz % n == 0; };
  a.wide = (wide(p->x, p->x_stride, size, 16) ? 1 : 0) | (wide(p->gate, p->gate_stride, size, 16) ? 2 : 0) |
           (wide(p->residual, p->residual_stride, size, 16) ? 4 : 0) |
           (wide(p->y, p->y_stride, osize, codes ? 8 : 16) ? 8 : 0) | (aligned(p->weight, 16) ? 16 : 0) |
           (aligned(p->next_weight, 16) ? 32 : 0);
  const BlockPick k = p->dtype == RSQ_BF16 ? pick_out<Bf16>(p->out_dtype, p->cols, p->rows)
                                            : pick_out<float>(p->out_dtype, p->cols, p->rows);
  // rows beyond what one launch may have go into further ones
  const int64_t most = max_blocks(k.threads) * k.rows, scales = p->scale_group ? p->cols / p->scale_group : 1;
  for (int64_t done = 0; done < p->rows; done += most) {
    a.rows = p->rows - done < most ? p->rows - done : most;
    a.x = static_cast<const uint8_t*>(p->x) + done * p->x_stride * size;
    if (p->gate) a.gate = static_cast<const uint8_t*>(p->gate) + done * p->gate_stride * size;
    if (p->residual) a.residual = static_cast<uint8_t*>(p->residual) + done * p->residual_stride * size;
    if (p->y) a.y = static_cast<uint8_t*>(p->y) + done * p->y_stride * osize;
    if (codes) a.scales = p->scales + done * scales;
    hipLaunchKernelGGL(k.fn, dim3((unsigned)ceil_div(a.rows, k.rows)), dim3(k.threads), 0, (hipStream_t)stream, a);
    if (const rsq_status s = launched("block norm")) return s;
  }
  return RSQ_OK;
}

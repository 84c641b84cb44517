// Root-mean-square norm of rows, with the residual's addition before it and an
// 8-bit output after it:
//   h = x + residual  (stored back, rounded to its type)
//   y = h / sqrt(mean(h^2) + eps) * weight
//   8 bits: per row or per `group` columns, scale = absmax(y) / qmax and
//   code = round(y / scale), nearest-even (int8: qmax 127; OCP E4M3: 448).
// The norm is taken of the fp32 sum, before h is rounded for the residual.
//
// Bound by memory: x and the residual are read once, the residual and the
// codes written once. A row stays in registers between its sums and its
// output: R threads own it, each kCols consecutive columns at a time, so that
// a wavefront reads 1 KB runs of bf16. 16384 x 4096 bf16 with a residual (537 MB)
// takes 98 us, 5.5 TB/s (a large copy, which misses the last-level cache more,
// moves 4.9); 16 rows of 2048 to E4M3 are 5.9 us of latency: launch, one round of
// loads, two sums.
#include <type_traits>

#include "host_util.hpp"
#include "norm.hpp"

namespace rsq {
namespace {

struct NormArgs {
  const void* x;
  void* residual;
  const float* weight;
  void* y;
  float* scales;
  int64_t x_stride, r_stride, y_stride;
  int64_t rows;
  int32_t cols, group;   // group 0: one scale a row
  float eps;
  int32_t wide;          // bit 0: x, 1: residual, 2: y, 3: weight take 16-byte (y: 8-byte codes) accesses
};

// R threads a row, up to NV * kCols columns a thread.
template <typename T, int OUT, int R, int NV>
__global__ __launch_bounds__(R < 256 ? 256 : R) void norm_kernel(NormArgs a) {
  constexpr int ROWS = R < 256 ? 256 / R : 1;
  __shared__ uint32_t lds[16];
  const int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / R;
  const int tid = threadIdx.x % R;
  // R < 256: a row belongs to one wavefront, nothing below crosses it
  if (row >= a.rows) return;
  const T* x = reinterpret_cast<const T*>(a.x) + row * a.x_stride;
  T* res = a.residual ? reinterpret_cast<T*>(a.residual) + row * a.r_stride : nullptr;
  float h[NV][kCols];
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) load_cols(x, (i * R + tid) * kCols, a.cols, a.wide & 1, h[i]);
  if (res) {
    float r[NV][kCols];
#pragma unroll
    for (int i = 0; i < NV; ++i) load_cols(res, (i * R + tid) * kCols, a.cols, a.wide & 2, r[i]);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int e = 0; e < kCols; ++e) h[i][e] += r[i][e];
      store_cols(res, (i * R + tid) * kCols, a.cols, a.wide & 2, h[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < kCols; ++e) sum = __builtin_fmaf(h[i][e], h[i][e], sum);
  sum = __uint_as_float(row_reduce<R, true>(__float_as_uint(sum), lds));
  const float rstd = 1.f / sqrtf(sum / (float)a.cols + a.eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float w[kCols];
    load_cols(a.weight, (i * R + tid) * kCols, a.cols, a.wide & 8, w);
#pragma unroll
    for (int e = 0; e < kCols; ++e) h[i][e] = h[i][e] * rstd * w[e];
  }
  store_row<OUT, R, NV>(h, a.y, a.scales, row, a.y_stride, a.cols, a.group, a.wide & 4, tid, lds);
}

typedef void (*NormFn)(NormArgs);
struct NormPick {
  NormFn fn;
  int threads, rows;
};

// A wavefront a row up to 1024 columns (its sums need no barrier), then 256, 512
// and 1024 threads, each with 8 to 32 columns: enough of a row in flight, and no
// thread without columns. 16384 rows of bf16 with a residual to bf16, us: 1024
// columns 21 (256 threads 27), 2048 40 (a wavefront 42, 512 threads 45), 4096 95
// (a wavefront 115, 1024 threads 125), 8192 186 (256 threads 195); 4096 rows of
// 16384 97 (512 threads 105). Four rows take 5 us with any of these.
template <typename T, int OUT>
NormPick pick(int cols) {
  if (cols <= 512) return {norm_kernel<T, OUT, 64, 1>, 256, 4};
  if (cols <= 1024) return {norm_kernel<T, OUT, 64, 2>, 256, 4};
  if (cols <= 2048) return {norm_kernel<T, OUT, 256, 1>, 256, 1};
  if (cols <= 4096) return {norm_kernel<T, OUT, 256, 2>, 256, 1};
  if (cols <= 8192) return {norm_kernel<T, OUT, 512, 2>, 512, 1};
  if (cols <= 16384) return {norm_kernel<T, OUT, 1024, 2>, 1024, 1};
  return {norm_kernel<T, OUT, 1024, 4>, 1024, 1};
}

template <typename T>
NormPick pick_out(int out, int cols) {
  switch (out) {
    case RSQ_F32: return pick<T, kOutF32>(cols);
    case RSQ_BF16: return pick<T, kOutBf16>(cols);
    case RSQ_INT8: return pick<T, kOutInt8>(cols);
    default: return pick<T, kOutE4m3>(cols);
  }
}

}  // namespace
}  // namespace rsq

using namespace rsq;

extern "C" rsq_status rsq_rms_norm(const rsq_norm* p, void* stream) {
  if (!p) return fail(RSQ_E_INVALID, "norm is NULL");
  if (p->dtype != RSQ_F32 && p->dtype != RSQ_BF16) return fail(RSQ_E_INVALID, "dtype %d", p->dtype);
  const bool codes = p->out_dtype == RSQ_INT8 || p->out_dtype == RSQ_E4M3;
  if (!codes && p->out_dtype != RSQ_F32 && p->out_dtype != RSQ_BF16)
    return fail(RSQ_E_INVALID, "out_dtype %d", p->out_dtype);
  if (p->rows < 0 || p->rows > 0x7fffffff || p->cols < 1)
    return fail(RSQ_E_INVALID, "rows %lld cols %d", (long long)p->rows, p->cols);
  if (p->cols > 32768) return fail(RSQ_E_UNSUPPORTED, "cols %d > 32768", p->cols);
  if (!(p->eps >= 0.f) || p->eps > 3.4e38f) return fail(RSQ_E_INVALID, "eps must be finite and >= 0");
  if (p->group != 0 && (!codes || (p->group != 32 && p->group != 64 && p->group != 128) || p->cols % p->group))
    return fail(RSQ_E_INVALID, "group %d: 0, or 32, 64 or 128 dividing cols %d with an 8-bit output", p->group, p->cols);
  if (p->rows == 0) return RSQ_OK;   // (an empty tensor has no address)
  if (codes != (p->scales != nullptr)) return fail(RSQ_E_INVALID, "scales are given with an 8-bit output, and only there");
  if (!p->x || !p->weight || !p->y) return fail(RSQ_E_INVALID, "x, weight and y must be non-NULL");
  if (p->x_stride < p->cols || p->y_stride < p->cols || (p->residual && p->residual_stride < p->cols))
    return fail(RSQ_E_INVALID, "a row stride is below %d columns", p->cols);
  const int size = p->dtype == RSQ_BF16 ? 2 : 4;
  const int osize = codes ? 1 : p->out_dtype == RSQ_BF16 ? 2 : 4;
  if (!aligned(p->x, size) || !aligned(p->residual, size) || !aligned(p->y, osize) || !aligned(p->weight, 4) ||
      !aligned(p->scales, 4))
    return fail(RSQ_E_INVALID, "a pointer is not aligned to its element type");
  const int64_t nscales = p->rows * (p->group ? p->cols / p->group : 1);
  const Span written[] = {{p->y, span_bytes(p->rows, p->y_stride, p->cols, osize), "y"},
                          {p->residual, span_bytes(p->rows, p->residual_stride, p->cols, size), "residual"},
                          {p->scales, nscales * 4, "scales"}};
  const Span read[] = {{p->x, span_bytes(p->rows, p->x_stride, p->cols, size), "x"},
                       {p->weight, (int64_t)p->cols * 4, "weight"}};
  if (const rsq_status s = check_overlap(written, read)) return s;

  NormArgs a{};
  a.weight = p->weight;
  a.x_stride = p->x_stride, a.r_stride = p->residual_stride, a.y_stride = p->y_stride;
  a.cols = p->cols, a.group = p->group, a.eps = p->eps;
  auto wide = [](const void* q, int64_t stride, int sz, int n) { return aligned(q, n) && stride * sz % n == 0; };
  a.wide = (wide(p->x, p->x_stride, size, 16) ? 1 : 0) |
           (p->residual && wide(p->residual, p->residual_stride, size, 16) ? 2 : 0) |
           (wide(p->y, p->y_stride, osize, codes ? 8 : 16) ? 4 : 0) | (aligned(p->weight, 16) ? 8 : 0);
  const NormPick k = p->dtype == RSQ_BF16 ? pick_out<Bf16>(p->out_dtype, p->cols) : pick_out<float>(p->out_dtype, p->cols);
  // rows beyond what one launch may have go into further ones
  const int64_t most = max_blocks(k.threads) * k.rows, scales = p->group ? p->cols / p->group : 1;
  for (int64_t done = 0; done < p->rows; done += most) {
    a.rows = p->rows - done < most ? p->rows - done : most;
    a.x = static_cast<const uint8_t*>(p->x) + done * p->x_stride * size;
    if (p->residual) a.residual = static_cast<uint8_t*>(p->residual) + done * p->residual_stride * size;
    a.y = static_cast<uint8_t*>(p->y) + done * p->y_stride * osize;
    if (codes) a.scales = p->scales + done * scales;
    hipLaunchKernelGGL(k.fn, dim3((unsigned)ceil_div(a.rows, k.rows)), dim3(k.threads), 0, (hipStream_t)stream, a);
    if (const rsq_status s = launched("RMS norm")) return s;
  }
  return RSQ_OK;
}

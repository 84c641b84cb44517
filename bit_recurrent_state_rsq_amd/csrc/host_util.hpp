// Host helpers shared by the C entry points: the thread's last error and the
// checks every operator call makes on its pointers.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "rsq.h"

namespace rsq {

// Record a message for rsq_last_error() and return `code`.
rsq_status fail(rsq_status code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
rsq_status hip_fail(hipError_t e, const char* what);

inline bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// A byte range [p, p + bytes) for the overlap check.
struct Span {
  const void* p;
  int64_t bytes;
  const char* name;
};

inline bool overlap(const Span& a, const Span& b) {
  if (!a.p || !b.p || a.bytes <= 0 || b.bytes <= 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + (uintptr_t)b.bytes && y < x + (uintptr_t)a.bytes;
}

// No written range may touch another written or a read one.
template <int NW, int NR>
rsq_status check_overlap(const Span (&written)[NW], const Span (&read)[NR]) {
  for (int i = 0; i < NW; ++i) {
    for (int j = 0; j < NR; ++j)
      if (overlap(written[i], read[j])) return fail(RSQ_E_INVALID, "%s overlaps %s", written[i].name, read[j].name);
    for (int j = i + 1; j < NW; ++j)
      if (overlap(written[i], written[j]))
        return fail(RSQ_E_INVALID, "%s overlaps %s", written[i].name, written[j].name);
  }
  return RSQ_OK;
}

// Bytes from the first to behind the last element of `rows` rows of `cols`
// elements, `stride` elements apart.
inline int64_t span_bytes(int64_t rows, int64_t stride, int64_t cols, int64_t size) {
  return rows > 0 ? ((rows - 1) * stride + cols) * size : 0;
}

inline rsq_status launched(const char* what) {
  const hipError_t e = hipGetLastError();
  return e == hipSuccess ? RSQ_OK : hip_fail(e, what);
}

// HIP takes launches of fewer than 2^32 threads along x: the most workgroups of
// `threads` that one launch may have.
constexpr int64_t max_blocks(int threads) { return 0xffffffffll / threads; }

// ... refused beyond
inline rsq_status check_blocks(int64_t blocks, int threads) {
  if (blocks <= max_blocks(threads)) return RSQ_OK;
  return fail(RSQ_E_UNSUPPORTED, "%lld workgroups of %d threads: 2^32 threads and more", (long long)blocks, threads);
}

}  // namespace rsq

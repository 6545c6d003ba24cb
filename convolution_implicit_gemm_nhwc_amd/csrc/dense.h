// What the host side of the dense operators shares: sizes and ranges of strided
// matrices.
#ifndef FCONV_DENSE_H
#define FCONV_DENSE_H

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace fconv {
namespace {

constexpr int64_t kMaxLd = 1 << 21;

__host__ __device__ inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
__host__ __device__ inline int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

inline hipStream_t as_stream(void* s) { return static_cast<hipStream_t>(s); }

inline bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  if (!a || !b || na == 0 || nb == 0) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
  return a0 < b0 + nb && b0 < a0 + na;
}
inline bool aligned(const void* ptr, uintptr_t n) { return (reinterpret_cast<uintptr_t>(ptr) & (n - 1)) == 0; }
// Bytes from the first to the last element of a strided matrix.
inline size_t span(int64_t rows, int64_t cols, int64_t ld, int es) {
  return rows <= 0 ? 0 : static_cast<size_t>((rows - 1) * ld + cols) * es;
}

struct Range {
  const void* p;
  size_t bytes;
};
// Whether any of the written ranges meets another range.
inline bool clash(const Range* out, int n_out, const Range* in, int n_in) {
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < n_in; ++j)
      if (overlaps(out[i].p, out[i].bytes, in[j].p, in[j].bytes)) return true;
    for (int j = i + 1; j < n_out; ++j)
      if (overlaps(out[i].p, out[i].bytes, out[j].p, out[j].bytes)) return true;
  }
  return false;
}

inline bool bad_ld(int64_t ld, int32_t D) { return ld < D || ld > kMaxLd; }

}  // namespace
}  // namespace fconv

#endif  // FCONV_DENSE_H

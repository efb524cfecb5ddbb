// Argument checks shared by the C ABI layers of the operators around the projections.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "bitlinear.h"

namespace bl {
namespace api {

inline bool aligned(const void* p, uintptr_t a) { return p && ((uintptr_t)p & (a - 1)) == 0; }
inline bool float_dtype(int d) { return d == BL_DTYPE_F32 || d == BL_DTYPE_BF16; }
inline int64_t esize(int d) { return d == BL_DTYPE_F32 ? 4 : d == BL_DTYPE_BF16 ? 2 : 1; }
inline int status_of(hipError_t e) { return e == hipSuccess ? BL_OK : BL_EIO; }

// A buffer of a call; NULL buffers do not take part.
struct Span {
  const void* p;
  uint64_t bytes;
};
inline bool overlap(const Span& a, const Span& b) {
  if (!a.p || !b.p || !a.bytes || !b.bytes) return false;
  const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
  return x < y + b.bytes && y < x + a.bytes;
}

// A launch holds fewer than 2^32 threads, and a row takes up to 1024 of them.
constexpr int64_t kMaxTokens = ((int64_t)1 << 22) - 1;
inline bool rows_ok(int64_t T, int64_t K) { return T >= 0 && T <= kMaxTokens && K >= 8 && K % 8 == 0; }

}  // namespace api
}  // namespace bl

// What the host sides of the operators check their arguments with.
#pragma once

#include <cuda_runtime.h>

#include <cstdarg>
#include <cstddef>
#include <cstdint>
#include <cstdio>

#include "xp.h"

namespace xp {
void set_last_error(const char* msg);

namespace checks {

inline xp_status fail(xp_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  try {
    xp::set_last_error(buf);
  } catch (...) {   // no memory for the message
  }
  return s;
}

#define XP_CUDA(call)                                                                     \
  do {                                                                                    \
    cudaError_t e_ = (call);                                                              \
    if (e_ != cudaSuccess) return fail(XP_ERR_CUDA, "%s: %s", #call, cudaGetErrorString(e_)); \
  } while (0)

inline bool is_float_type(int dt) { return dt == XP_F32 || dt == XP_BF16; }
inline size_t size_of(int dt) { return dt == XP_F32 ? 4 : dt == XP_BF16 ? 2 : 1; }
inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
inline size_t round_up(size_t a, size_t b) { return (a + b - 1) / b * b; }

inline xp_status check_rows(const char* what, const void* p, size_t stride, size_t rows, size_t cols, int dtype) {
  if (!p) return fail(XP_ERR_INVALID, "%s is NULL", what);
  if (stride < cols && rows > 1) return fail(XP_ERR_INVALID, "%s: rows %zu elements apart overlap (%zu columns)", what, stride, cols);
  if (stride > ((size_t)1 << 40)) return fail(XP_ERR_INVALID, "%s: rows %zu elements apart", what, stride);
  if (!aligned(p, size_of(dtype))) return fail(XP_ERR_INVALID, "%s is not aligned to its element", what);
  return XP_OK;
}

// Where a matrix of `rows` rows lies.
struct Span {
  uintptr_t lo, hi;
  size_t rows, width, pitch;   // bytes of a row, and from one row to the next
};
inline Span span_of(const void* p, size_t stride, size_t rows, size_t cols, size_t es) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return {lo, lo + ((rows - 1) * stride + cols) * es, rows, cols * es, stride * es};
}
// Whether two matrices share bytes.  At equal strides rows may
// lie between rows, as side-by-side columns of one buffer do: b's rows begin at
// the same place between two of a's.  At different strides that is not followed up.
inline bool overlap(const Span& a, const Span& b) {
  if (a.hi <= b.lo || b.hi <= a.lo) return false;
  if (a.rows == 1 || a.pitch != b.pitch) return true;
  const size_t at = b.lo >= a.lo ? (b.lo - a.lo) % a.pitch : (a.pitch - (a.lo - b.lo) % a.pitch) % a.pitch;
  return at < a.width || a.pitch - at < b.width;
}
inline bool same(const Span& a, const Span& b) { return a.lo == b.lo && (a.rows == 1 || a.pitch == b.pitch); }

}  // namespace checks
}  // namespace xp

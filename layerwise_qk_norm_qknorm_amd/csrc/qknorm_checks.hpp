// Host-side argument checks and error strings shared by the C ABI files of
// libqknorm.so. Plain C++ with no HIP call.
#pragma once

#include <stdint.h>

#include <cstdarg>
#include <cstdio>
#include <string>

#include "qknorm.h"

namespace qkn {

inline thread_local std::string g_last_error;  // the per-thread message of qknorm_last_error

inline int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  g_last_error = buf;
  return code;
}

inline int ok() {
  g_last_error.clear();
  return QKNORM_OK;
}

inline size_t elem_size(int dtype) {
  if (dtype == QKNORM_F32) return 4;
  if (dtype == QKNORM_BF16) return 2;
  if (dtype == QKNORM_FP8_E4M3) return 1;
  return 0;
}

// gamma is bf16 for FP8 rows, the row type otherwise
inline size_t gamma_size(int dtype) { return dtype == QKNORM_F32 ? 4 : 2; }

// The set of bytes touched by rows t < T, columns j < h of a strided matrix.
struct Region {
  uintptr_t base;
  int64_t ld;   // elements
  int64_t h;    // elements
  int64_t T;
  int64_t esz;  // bytes per element
  int64_t span_bytes() const { return ((T - 1) * ld + h) * esz; }
};

// True if the two element sets may share a byte. Exact for equal strides and
// element sizes (the packed-QKV case); conservative (byte spans) otherwise.
inline bool may_overlap(const Region& a, const Region& b) {
  if (a.T <= 0 || b.T <= 0 || a.h <= 0 || b.h <= 0) return false;
  const uintptr_t a0 = a.base, a1 = a.base + (uintptr_t)a.span_bytes();
  const uintptr_t b0 = b.base, b1 = b.base + (uintptr_t)b.span_bytes();
  if (a1 <= b0 || b1 <= a0) return false;
  if (a.ld != b.ld || a.esz != b.esz || a.T == 1 || b.T == 1) return true;
  const int64_t d = (int64_t)(b.base - a.base);  // may be negative
  if (d % a.esz != 0) return true;
  const int64_t de = d / a.esz;
  // Column of a's row grid where b's rows start.
  const int64_t r = ((de % a.ld) + a.ld) % a.ld;
  if (r + b.h <= a.ld) return r < a.h;                  // b occupies [r, r + b.h)
  return true;                                          // b wraps into a's next row
}

inline bool same_region(const Region& a, const Region& b) {
  return a.base == b.base && a.ld == b.ld && a.h == b.h && a.esz == b.esz;
}

inline bool fits(int64_t T, int64_t ld, int64_t h, int64_t esz) {
  // (T - 1) * ld + h elements, times esz bytes, must fit in int64.
  if (T <= 0) return true;
  const int64_t lim = INT64_MAX / esz;
  if (T - 1 > 0 && ld > (lim - h) / (T - 1)) return false;
  return true;
}

}  // namespace qkn

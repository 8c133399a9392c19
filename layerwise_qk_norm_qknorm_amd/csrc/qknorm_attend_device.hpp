// Device helpers shared by the attention kernels (qknorm_attend.hip,
// qknorm_attend_wide.hip): which tokens a query row sees, page lookups, and the
// running maximum of a row's scores.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qknorm_device.hpp"
#include "qknorm_internal.hpp"
#include "qknorm_ops.hpp"

namespace qkn {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));

// A row's reference maximum follows its scores only when they pass it by 2^8:
// float32 sums and bf16 probabilities keep their relative accuracy at any
// scale, and the accumulator is hardly ever rescaled.
constexpr float kSlack = 8.0f;
// The reference before any score: the lowest finite value, so that every score
// that is finite in base 2 (times log2 e) counts. Differences to it may be
// infinite, never NaN.
constexpr float kNothing = -3.40282347e38f;

struct Frag {
  uint32_t w[4];
  __device__ __forceinline__ bf16x8_t get() const { return __builtin_bit_cast(bf16x8_t, *this); }
};

// The largest of three, NaN where one of them is: one v_maximum3_f32. (fmaxf
// would spend an instruction per operand on quieting NaNs. Written as inline
// asm it would read the scores without the wait states that a matrix product's
// result needs, which the compiler puts only before instructions it knows.) A
// row with a NaN score is NaN whatever its maximum.
__device__ __forceinline__ float max3(float a, float b, float c) {
  return __builtin_elementwise_maximum(__builtin_elementwise_maximum(a, b), c);
}

// In a branch that few tiles take: keeps the compiler from running it for all
// of them as selects (the edge masks alone are 96 instructions of a tile).
__device__ __forceinline__ void keep_branch() { asm volatile(""); }

__device__ __forceinline__ float row_max(float v) {   // over the four lanes that hold a row
  auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = max3(__uint_as_float(p[0]), __uint_as_float(p[1]), __uint_as_float(p[1]));
  p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return max3(__uint_as_float(p[0]), __uint_as_float(p[1]), __uint_as_float(p[1]));
}

// A sequence's query rows and cached length, held to what the arrays hold.
struct Sequence {
  int q0, nq, len;
};
__device__ __forceinline__ Sequence sequence(const AttendArgs& a, int b) {
  Sequence s{b, 1, load_uniform(a.seq_lens + b)};
  if (a.cu_q) {
    const int q0 = load_uniform(a.cu_q + b), q1 = load_uniform(a.cu_q + b + 1);
    s.q0 = q0 < 0 ? 0 : q0 > a.T ? a.T : q0;
    s.nq = (q1 < s.q0 ? s.q0 : q1 > a.T ? a.T : q1) - s.q0;
  }
  s.len = s.len < 0 ? 0 : s.len > a.table_tokens ? a.table_tokens : s.len;
  return s;
}
// Tokens [lo, hi) that query i of a sequence sees.
__device__ __forceinline__ int see_hi(const AttendArgs& a, const Sequence& s, int i) {
  const int pos = s.len - s.nq + i;
  return pos < 0 ? 0 : a.causal ? pos + 1 : s.len;
}
__device__ __forceinline__ int see_lo(const AttendArgs& a, const Sequence& s, int i) {
  const int lo = s.len - s.nq + i - a.window + 1;
  return a.window && lo > 0 ? lo : 0;
}
// A block's rows r0 .. : what they see together, and the chunks that takes.
struct Span {
  int first, hi;     // first: a multiple of 32
  int chunks;
};
__device__ __forceinline__ Span span(const AttendArgs& a, const Sequence& s, int i_first, int i_last) {
  Span p;
  const int lo = see_lo(a, s, i_first);
  p.hi = see_hi(a, s, i_last);
  p.first = lo & ~31;
  p.chunks = p.hi > lo ? (int)((uint32_t)(p.hi - p.first + a.chunk - 1) / (uint32_t)a.chunk) : 0;
  return p;
}

}  // namespace
}  // namespace qkn

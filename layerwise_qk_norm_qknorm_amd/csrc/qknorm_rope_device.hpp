// Device helpers shared by the kernels that normalize, rotate and store heads
// (qknorm_rope.hip, qknorm_rope_paired.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qknorm_device.hpp"
#include "qknorm_internal.hpp"
#include "qknorm_ops.hpp"

namespace qkn {
namespace {

typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));

// BYTES bytes at p (aligned to min(BYTES, 16)) into words; smaller elements
// land in the low bits of the first word.
template <int BYTES, bool STREAM>
__device__ __forceinline__ void load_bytes(const char* p, uint32_t* w) {
  if constexpr (BYTES >= 16) {
#pragma unroll
    for (int q = 0; q < BYTES / 16; ++q) {
      const u32x4_t* src = reinterpret_cast<const u32x4_t*>(p) + q;
      const u32x4_t v = STREAM ? __builtin_nontemporal_load(src) : *src;
      w[4 * q] = v.x;
      w[4 * q + 1] = v.y;
      w[4 * q + 2] = v.z;
      w[4 * q + 3] = v.w;
    }
  } else if constexpr (BYTES == 8) {
    const u32x2_t v = *reinterpret_cast<const u32x2_t*>(p);
    w[0] = v.x;
    w[1] = v.y;
  } else if constexpr (BYTES == 4) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (BYTES == 2) {
    w[0] = *reinterpret_cast<const uint16_t*>(p);
  } else {
    w[0] = *reinterpret_cast<const uint8_t*>(p);
  }
}

template <int BYTES>
__device__ __forceinline__ void store_bytes(char* p, const uint32_t* w) {
  if constexpr (BYTES == 16) {
    const u32x4_t v = {w[0], w[1], w[2], w[3]};
    __builtin_nontemporal_store(v, reinterpret_cast<u32x4_t*>(p));
  } else if constexpr (BYTES == 8) {
    const u32x2_t v = {w[0], w[1]};
    *reinterpret_cast<u32x2_t*>(p) = v;
  } else if constexpr (BYTES == 4) {
    *reinterpret_cast<uint32_t*>(p) = w[0];
  } else if constexpr (BYTES == 2) {
    *reinterpret_cast<uint16_t*>(p) = (uint16_t)w[0];
  } else {
    *reinterpret_cast<uint8_t*>(p) = (uint8_t)w[0];
  }
}

template <int BYTES>
struct Piece {
  uint32_t w[BYTES >= 4 ? BYTES / 4 : 1];
};

// A piece of row data as float32 (exact).
template <class IO, int VW>
__device__ __forceinline__ void widen(const uint32_t* w, float (&v)[VW]) {
  if constexpr (IO::kBytes == 4) {
#pragma unroll
    for (int e = 0; e < VW; ++e) v[e] = __uint_as_float(w[e]);
  } else if constexpr (IO::kBytes == 2) {
#pragma unroll
    for (int e = 0; e < VW; ++e) v[e] = (e & 1) ? bf16_hi(w[e >> 1]) : bf16_lo(w[e >> 1]);
  } else if constexpr (VW == 1) {
    v[0] = __builtin_amdgcn_cvt_pk_f32_fp8(w[0], false)[0];
  } else {
#pragma unroll
    for (int p = 0; p < VW / 4; ++p) {
      const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8(w[p], false);
      const f32x2_t hi = __builtin_amdgcn_cvt_pk_f32_fp8(w[p], true);
      v[4 * p] = lo[0];
      v[4 * p + 1] = lo[1];
      v[4 * p + 2] = hi[0];
      v[4 * p + 3] = hi[1];
    }
  }
}

// gamma of a piece as float32: bf16, or float32 for float32 rows.
template <class IO, int VW>
__device__ __forceinline__ void widen_gamma(const uint32_t* w, float (&v)[VW]) {
#pragma unroll
  for (int e = 0; e < VW; ++e)
    v[e] = IO::kGBytes == 4 ? __uint_as_float(w[e]) : (e & 1) ? bf16_hi(w[e >> 1]) : bf16_lo(w[e >> 1]);
}

// In a branch that few waves take: keeps the compiler from running it for all
// of them as selects.
__device__ __forceinline__ void keep_branch() { asm volatile(""); }

// float32 -> a piece of the row type, one rounding to nearest even (FP8
// saturates to +-448, NaN stays NaN).
template <class IO, int VW>
__device__ __forceinline__ void narrow(const float (&v)[VW], uint32_t* w) {
  if constexpr (IO::kBytes == 4) {
#pragma unroll
    for (int e = 0; e < VW; ++e) w[e] = __float_as_uint(v[e]);
  } else if constexpr (IO::kBytes == 2) {
    if constexpr (VW == 1) {
      const f32x2_t f = {v[0], 0.0f};
      w[0] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2_t));
    } else {
#pragma unroll
      for (int p = 0; p < VW / 2; ++p) {
        const f32x2_t f = {v[2 * p], v[2 * p + 1]};
        w[p] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2_t));
      }
    }
  } else if constexpr (VW == 1) {
    w[0] = pack_fp8_word(sat_e4m3(v[0]), 0.0f, 0.0f, 0.0f);
  } else {
    // saturating costs four operations a value; the largest magnitude (NaN
    // above all) costs half of one, and tells whether any needs it
    float big = 0.0f;
#pragma unroll
    for (int e = 0; e < VW; e += 2)
      big = __builtin_elementwise_maximum(__builtin_elementwise_maximum(big, __builtin_fabsf(v[e])),
                                          __builtin_fabsf(v[e + 1]));
    if (__builtin_amdgcn_ballot_w64(!(big <= 448.0f)) != 0) {
      keep_branch();
#pragma unroll
      for (int p = 0; p < VW / 4; ++p)
        w[p] = pack_fp8_word(sat_e4m3(v[4 * p]), sat_e4m3(v[4 * p + 1]), sat_e4m3(v[4 * p + 2]),
                             sat_e4m3(v[4 * p + 3]));
    } else {
#pragma unroll
      for (int p = 0; p < VW / 4; ++p) w[p] = pack_fp8_word(v[4 * p], v[4 * p + 1], v[4 * p + 2], v[4 * p + 3]);
    }
  }
}

// A wave's tokens t, t + step, ...: each token's loads are issued before the
// one before it is worked on, in two buffers that take turns. The loop loads
// without a condition (past the last token, that one again): a branch around
// the loads would make the waits hold for both ways, and so wait for all. A
// wave of one token loads it alone.
template <class In, class Load, class Work>
__device__ __forceinline__ void each_token(int64_t t, int64_t step, int64_t T, const Load& load, const Work& work) {
  if (t >= T) return;
  In one;
  load(one, t);
  if (t + step >= T) {
    work(one, t);
    return;
  }
  In two;
  while (true) {
    load(two, t + step < T ? t + step : t);
    work(one, t);
    t += step;
    if (t >= T) break;
    load(one, t + step < T ? t + step : t);
    work(two, t);
    t += step;
    if (t >= T) break;
  }
}

// float64 sums over a head's lanes, by the same steps as group_sum.
template <int CTRL>
__device__ __forceinline__ double dpp_move_d(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)u, CTRL, 0xF, 0xF, false);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(u >> 32), CTRL, 0xF, 0xF, false);
  return __builtin_bit_cast(double, ((uint64_t)hi << 32) | lo);
}
__device__ __forceinline__ double swap_add_d(double v, bool across32) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)u, hi = (uint32_t)(u >> 32);
  const auto l = across32 ? __builtin_amdgcn_permlane32_swap(lo, lo, false, false)
                          : __builtin_amdgcn_permlane16_swap(lo, lo, false, false);
  const auto h = across32 ? __builtin_amdgcn_permlane32_swap(hi, hi, false, false)
                          : __builtin_amdgcn_permlane16_swap(hi, hi, false, false);
  return __builtin_bit_cast(double, ((uint64_t)h[0] << 32) | l[0]) +
         __builtin_bit_cast(double, ((uint64_t)h[1] << 32) | l[1]);
}
__device__ __forceinline__ double group_sum_d(double v, int group) {
  if (group > 1) v += dpp_move_d<0xB1>(v);
  if (group > 2) v += dpp_move_d<0x4E>(v);
  if (group > 4) v += dpp_move_d<0x141>(v);
  if (group > 8) v += dpp_move_d<0x140>(v);
  if (group > 16) v = swap_add_d(v, false);
  if (group > 32) v = swap_add_d(v, true);
  return v;
}

// float64 -> float32 rounded to odd: truncated, and the last bit set if
// anything was lost. Rounding that once more to a format of at least two bits
// fewer gives what rounding the float64 value once would have given.
__device__ __forceinline__ float round_to_odd(double z) {
  const float f = (float)z;
  const double back = (double)f;
  uint32_t u = __float_as_uint(f);
  if (__builtin_fabs(back) > __builtin_fabs(z)) u -= 1;      // toward zero (infinity: to the largest)
  if (back != z && z == z) u |= 1;
  return __uint_as_float(u);
}

}  // namespace
}  // namespace qkn

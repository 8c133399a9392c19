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

// Positions on several axes. A wave gathers its token's angles, a lane's each
// (lane + 64 r), from the rows that their axes' positions name, and lays them side
// by side in LDS, where its lanes then read them as they would a row of the table:
// two loads of 4 bytes a lane instead of its chunk's angles for each lane, whatever
// the order of the axes (8192 tokens of 40 + 8 bf16 heads of 128: sections 43.2 us
// with each lane's own loads, 38.7 so; axes in turn 63 and 39.4; a single position,
// loaded as chunks, 36.6).
// Angles past the first 128 are gathered when they are laid down, so that they
// take no registers (rotations of more than 256 columns).
constexpr int kSinAt(int rounds) { return 64 * rounds; }     // floats; rounds: 64 angles each
constexpr int kHeldRounds = 2;
struct AxisAngles {
  float c[kHeldRounds], s[kHeldRounds];
  uint32_t lost;       // bits of the angles whose position lies outside the table: NaN

  struct Rows {        // (in an array they would be chosen from in memory)
    uint64_t row0, row1, row2, row3;
    uint32_t in;
  };
  static_assert(kMostAxes == 4, "Rows");
  struct Positions {
    int64_t on[kMostAxes];      // axes there are not: the first one's
    template <class Args>
    __device__ __forceinline__ void load(const Args& a, int64_t t) {
#pragma unroll
      for (int x = 0; x < kMostAxes; ++x) on[x] = load_uniform(a.positions + (x < a.axes.n ? x : 0) * a.axes.ld + t);
    }
  };
  template <class Args>
  __device__ __forceinline__ static Rows rows(const Args& a, const Positions& pos) {
    Rows w;
    w.in = 0;
    const auto row = [&](int x) {
      const bool ok = pos.on[x] >= 0 && pos.on[x] < a.n_positions;
      w.in |= (uint32_t)ok << x;
      return uniform64(reinterpret_cast<uint64_t>(a.cos_sin + (ok ? pos.on[x] : 0) * a.ld_table));
    };
    w.row0 = row(0), w.row1 = row(1), w.row2 = row(2), w.row3 = row(3);
    return w;
  }
  // Angle j (past the last: the first), on axis x.
  __device__ __forceinline__ static bool fetch(const Rows& w, uint32_t x, int j, int half, float& c, float& s) {
    const uint64_t lo = x & 1 ? w.row1 : w.row0, hi = x & 1 ? w.row3 : w.row2;
    const float* p = reinterpret_cast<const float*>(x & 2 ? hi : lo) + (j < half ? j : 0);
    c = p[0];
    s = p[half];
    return w.in >> x & 1;
  }
  // axis: lane_axes
  template <class Args>
  __device__ __forceinline__ void load(const Args& a, const Positions& pos, uint32_t axis) {
    const Rows w = rows(a, pos);
    const int half = a.rot >> 1, lane = threadIdx.x & 63;
    lost = 0;
#pragma unroll
    for (int r = 0; r < kHeldRounds; ++r) {
      c[r] = s[r] = 0.0f;
      if (64 * r < half) lost |= (uint32_t)!fetch(w, axis >> (2 * r) & 3, lane + 64 * r, half, c[r], s[r]) << r;
    }
  }
  template <int ROUNDS, class Args>
  __device__ __forceinline__ void put(const Args& a, int64_t t, float* lds) const {
    const int half = a.rot >> 1, lane = threadIdx.x & 63;
    const float nan = __builtin_nanf("");
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int r = 0; r < kHeldRounds; ++r)
      if (r < ROUNDS && 64 * r < half) {
        lds[lane + 64 * r] = lost >> r & 1 ? nan : c[r];
        lds[kSinAt(ROUNDS) + lane + 64 * r] = lost >> r & 1 ? nan : s[r];
      }
    if (ROUNDS > kHeldRounds && half > 64 * kHeldRounds) {
      keep_branch();
      Positions pos;
      pos.load(a, t);
      const Rows w = rows(a, pos);
#pragma unroll 1
      for (int j = lane + 64 * kHeldRounds; j - lane < half; j += 64) {
        float cj, sj;
        const bool in = fetch(w, a.axes.of[j >> 4] >> (2 * (j & 15)) & 3, j, half, cj, sj);
        lds[j] = in ? cj : nan;
        lds[kSinAt(ROUNDS) + j] = in ? sj : nan;
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
  }
};
// The axes of a lane's held angles, two bits each (arguments without axes: none).
__device__ __forceinline__ uint32_t lane_axes(const RopeArgs&) { return 0; }
__device__ __forceinline__ uint32_t lane_axes(const RopeGradArgs&) { return 0; }
template <class Args>
__device__ __forceinline__ uint32_t lane_axes(const Args& a) {
  const RopeAxes& axes = a.axes;
  uint32_t own = 0;
#pragma unroll
  for (int r = 0; r < kHeldRounds; ++r) {
    const int j = (threadIdx.x & 63) + 64 * r;
    own |= (axes.of[j >> 4] >> (2 * (j & 15)) & 3) << (2 * r);
  }
  return own;
}

// The formats of quantised caches. A block of 32 channels has the scale 2^E, E =
// floor(log2(largest magnitude)) - kLead held to [-100, kTop - 127], and codes
// rounded to nearest even, magnitudes past the largest code's saturating. One
// that holds an infinity or NaN gets codes 0 and the scale byte 0xFF and reads as
// NaN. kMostFactor: see qknorm_rope_rows.
struct Mx4 {   // E2M1
  static constexpr int kBits = 4, kLead = 2, kTop = 252;
  static constexpr float kMostFactor = 0x1p24f;
  __device__ __forceinline__ static float saturated(float v) { return v; }   // by the conversion
};
struct Mx8 {   // E4M3
  static constexpr int kBits = 8, kLead = 8, kTop = 246;
  static constexpr float kMostFactor = 0x1p16f;
  // the conversion makes NaN of what it would round to more than 448
  __device__ __forceinline__ static float saturated(float v) { return __builtin_amdgcn_fmed3f(v, -448.0f, 448.0f); }
};

// The scale byte of a block whose largest magnitude has these bits (NaN above infinity).
template <class MX>
__device__ __forceinline__ int scale_byte(uint32_t m) {
  return m >= 0x7F800000u ? 0xFF : min(max((int)(m >> 23) - MX::kLead, 27), MX::kTop);
}
__device__ __forceinline__ float over_scale(int byte) {   // 2^-E
  return __uint_as_float((uint32_t)(254 - (byte == 0xFF ? 127 : byte)) << 23);
}
template <class MX, int VW>
struct Codes {
  uint32_t w[VW * MX::kBits / 32 > 0 ? VW * MX::kBits / 32 : 1];
  __device__ __forceinline__ bool operator==(const Codes& o) const {
    bool same = true;
#pragma unroll
    for (uint32_t i = 0; i < sizeof(w) / 4; ++i) same = same && w[i] == o.w[i];
    return same;
  }
};
// The codes of values already over the scale and saturated (as MX::saturated, or less than
// half a step past the largest code).
template <class MX, int VW>
__device__ __forceinline__ Codes<MX, VW> codes_of(const float (&a)[VW]) {
  Codes<MX, VW> q;
  if constexpr (MX::kBits == 4) {
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, a[0], a[1], 1.0f, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, a[2], a[3], 1.0f, 1);
    if constexpr (VW == 8) {
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, a[4], a[5], 1.0f, 2);
      w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, a[6], a[7], 1.0f, 3);
    }
    q.w[0] = w;
  } else {
#pragma unroll
    for (int p = 0; p < VW / 4; ++p) q.w[p] = pack_fp8_word(a[4 * p], a[4 * p + 1], a[4 * p + 2], a[4 * p + 3]);
  }
  return q;
}
// What a block's scale byte stands for: 2^(byte - 127), for bytes up to 254. The exponent
// field of 0 is subnormal: 2^-127 has the bits 0x00400000.
__device__ __forceinline__ float scale_value(uint32_t byte) { return __uint_as_float(max(byte << 23, 0x00400000u)); }
// The values that codes with a scale byte stand for (exact).
template <class MX, int VW>
__device__ __forceinline__ void code_values(const Codes<MX, VW>& q, int byte, float (&f)[VW]) {
  const float back = byte == 0xFF ? __builtin_nanf("") : scale_value(byte);
  if constexpr (MX::kBits == 4) {
    const f32x2_t y0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q.w[0], 1.0f, 0);
    const f32x2_t y1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q.w[0], 1.0f, 1);
    f[0] = y0[0] * back, f[1] = y0[1] * back, f[2] = y1[0] * back, f[3] = y1[1] * back;
    if constexpr (VW == 8) {
      const f32x2_t y2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q.w[0], 1.0f, 2);
      const f32x2_t y3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q.w[0], 1.0f, 3);
      f[4] = y2[0] * back, f[5] = y2[1] * back, f[6] = y3[0] * back, f[7] = y3[1] * back;
    }
  } else {
#pragma unroll
    for (int p = 0; p < VW / 4; ++p) {
      const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8(q.w[p], false);
      const f32x2_t hi = __builtin_amdgcn_cvt_pk_f32_fp8(q.w[p], true);
      f[4 * p] = lo[0] * back, f[4 * p + 1] = lo[1] * back, f[4 * p + 2] = hi[0] * back, f[4 * p + 3] = hi[1] * back;
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

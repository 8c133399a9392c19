// Device helpers shared by the kernels of libqknorm.so: I/O types, 16-byte
// chunk loads and stores, conversions, lane sums and the RMS factor.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "qknorm_internal.hpp"
#include "qknorm_ops.hpp"

namespace qkn {
namespace {

// I/O types. kVW: elements per 16-byte row chunk; kBytes: bytes per row
// element; kGW / kGBytes: 32-bit words of gamma per chunk and bytes per gamma
// element (FP8 rows take bf16 gamma).
struct BF16 {
  static constexpr int kVW = 8, kBytes = 2, kGW = 4, kGBytes = 2, kDtype = kDtypeBF16;
};
struct F32 {
  static constexpr int kVW = 4, kBytes = 4, kGW = 4, kGBytes = 4, kDtype = kDtypeF32;
};
struct FP8 {  // OCP FP8 E4M3 (E4M3FN) rows, bf16 gamma
  static constexpr int kVW = 16, kBytes = 1, kGW = 8, kGBytes = 2, kDtype = kDtypeFP8;
};

template <int W>
struct Words {
  uint32_t w[W];
};
using Chunk = Words<4>;  // 16 bytes of row data
template <class IO>
using GChunk = Words<IO::kGW>;  // the gamma of one chunk

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x2_t __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4_t __attribute__((ext_vector_type(4)));

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// All elements of a row chunk as float32 (exact widening).
template <class IO>
__device__ __forceinline__ void decode(const Chunk& c, float (&v)[IO::kVW]);
template <>
__device__ __forceinline__ void decode<BF16>(const Chunk& c, float (&v)[8]) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    v[2 * p] = bf16_lo(c.w[p]);
    v[2 * p + 1] = bf16_hi(c.w[p]);
  }
}
template <>
__device__ __forceinline__ void decode<F32>(const Chunk& c, float (&v)[4]) {
#pragma unroll
  for (int p = 0; p < 4; ++p) v[p] = __uint_as_float(c.w[p]);
}
template <>
__device__ __forceinline__ void decode<FP8>(const Chunk& c, float (&v)[16]) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {  // v_cvt_pk_f32_fp8: two E4M3 values of one 16-bit half per instruction
    const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8(c.w[p], false);
    const f32x2_t hi = __builtin_amdgcn_cvt_pk_f32_fp8(c.w[p], true);
    v[4 * p] = lo[0];
    v[4 * p + 1] = lo[1];
    v[4 * p + 2] = hi[0];
    v[4 * p + 3] = hi[1];
  }
}

// The gamma of a chunk as float32 (exact).
template <class IO>
__device__ __forceinline__ void decode_gamma(const GChunk<IO>& g, float (&v)[IO::kVW]) {
  if (IO::kGBytes == 2) {
#pragma unroll
    for (int p = 0; p < IO::kGW; ++p) {
      v[2 * p] = bf16_lo(g.w[p]);
      v[2 * p + 1] = bf16_hi(g.w[p]);
    }
  } else {
#pragma unroll
    for (int p = 0; p < IO::kGW; ++p) v[p] = __uint_as_float(g.w[p]);
  }
}

// float32 results -> a chunk of the I/O type, one rounding to nearest even.
// For FP8 the caller saturates to +-448 first where needed (sat_e4m3; NaN
// stays NaN): the hardware conversion turns magnitudes past 464 into NaN.
template <class IO>
__device__ __forceinline__ void pack(Chunk& c, const float (&v)[IO::kVW]);
template <>
__device__ __forceinline__ void pack<BF16>(Chunk& c, const float (&v)[8]) {
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    const f32x2_t f = {v[2 * p], v[2 * p + 1]};
    c.w[p] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2_t));
  }
}
template <>
__device__ __forceinline__ void pack<F32>(Chunk& c, const float (&v)[4]) {
#pragma unroll
  for (int p = 0; p < 4; ++p) c.w[p] = __float_as_uint(v[p]);
}
__device__ __forceinline__ float sat_e4m3(float x) { return x > 448.0f ? 448.0f : (x < -448.0f ? -448.0f : x); }
// Four float32 values -> four E4M3 codes in one word, each conversion
// filling one 16-bit half. The first one's word operand (the half it keeps)
// is its own first input, dead afterwards, instead of a zeroed register: the
// second conversion overwrites that half anyway, and no move is needed.
__device__ __forceinline__ uint32_t pack_fp8_word(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, __float_as_int(a), false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
  return (uint32_t)w;
}
template <>
__device__ __forceinline__ void pack<FP8>(Chunk& c, const float (&v)[16]) {
#pragma unroll
  for (int p = 0; p < 4; ++p) c.w[p] = pack_fp8_word(v[4 * p], v[4 * p + 1], v[4 * p + 2], v[4 * p + 3]);
}

// Loads `W` words at `p`: 16-byte loads (p 16-byte aligned) on the aligned
// path; on the element-wise path the first `n` elements of `esz` bytes, the
// rest reading as 0.
//
// Every load is unconditional: a lane whose slot is idle passes the row's
// first chunk (always a valid address) and its value is masked by the caller.
// Predicated loads would put each load in its own branch with a wait for it
// before the join, leaving one load in flight per wave.
template <int W, int ESZ, bool ALIGNED>
__device__ __forceinline__ Words<W> load_words(const char* p, int n) {
  Words<W> c;
#pragma unroll
  for (int q = 0; q < W; ++q) c.w[q] = 0u;
  if (ALIGNED) {
#pragma unroll
    for (int q = 0; q < W; q += 4) {
      const u32x4_t v = *reinterpret_cast<const u32x4_t*>(p + 4 * q);
      c.w[q] = v.x;
      c.w[q + 1] = v.y;
      c.w[q + 2] = v.z;
      c.w[q + 3] = v.w;
    }
  } else {
    constexpr int kElems = W * 4 / ESZ;
#pragma unroll
    for (int e = 0; e < kElems; ++e) {
      const int ee = e < n ? e : 0;
      uint32_t v;
      if (ESZ == 1) v = reinterpret_cast<const uint8_t*>(p)[ee];
      else if (ESZ == 2) v = reinterpret_cast<const uint16_t*>(p)[ee];
      else v = reinterpret_cast<const uint32_t*>(p)[ee];
      c.w[(e * ESZ) / 4] |= (e < n ? v : 0u) << (((e * ESZ) % 4) * 8);
    }
  }
  return c;
}

// The chunk at element offset `col` of row `row` (the first `n` elements on
// the element-wise path). Row data is read once, so the 16-byte path marks
// the loads non-temporal, as the stores are (gamma and the statistics, read
// by many blocks, keep ordinary loads). Measured on MI355X against ordinary
// loads, alternated on one box with identical outputs: GQA prefill fused
// 34.92 -> 34.20 us, FP8 rows 20.20 -> 19.88 us, headwise 34.18 -> 32.95 us,
// rank-slice apply 18.96 -> 18.62 us, 256-token decode rows 4.41 -> 3.84 us.
template <class IO, bool ALIGNED>
__device__ __forceinline__ Chunk load_chunk(const char* row, int col, int n) {
  if constexpr (ALIGNED) {
    const u32x4_t v = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(row + (int64_t)col * IO::kBytes));
    Chunk c;
    c.w[0] = v.x;
    c.w[1] = v.y;
    c.w[2] = v.z;
    c.w[3] = v.w;
    return c;
  }
  return load_words<4, IO::kBytes, ALIGNED>(row + (int64_t)col * IO::kBytes, n);
}

// The gamma of the chunk at column `col`, from gamma base `base`.
template <class IO, bool ALIGNED>
__device__ __forceinline__ GChunk<IO> load_gamma(const char* base, int col, int n) {
  return load_words<IO::kGW, IO::kGBytes, ALIGNED>(base + (int64_t)col * IO::kGBytes, n);
}

// Stores the first `n` elements of a chunk. Results are written once and not
// read again by this kernel, so the 16-byte path marks them non-temporal
// (streamed past the caches), which measured faster on MI355X.
template <class IO, bool ALIGNED>
__device__ __forceinline__ void store_chunk(char* row, int col, int n, const Chunk& c) {
  char* p = row + (int64_t)col * IO::kBytes;
  if (ALIGNED) {
    const u32x4_t v = {c.w[0], c.w[1], c.w[2], c.w[3]};
    __builtin_nontemporal_store(v, reinterpret_cast<u32x4_t*>(p));
  } else {
#pragma unroll
    for (int e = 0; e < IO::kVW; ++e) {
      if (e < n) {
        const uint32_t v = c.w[(e * IO::kBytes) / 4] >> (((e * IO::kBytes) % 4) * 8);
        if (IO::kBytes == 1) reinterpret_cast<uint8_t*>(p)[e] = (uint8_t)v;
        else if (IO::kBytes == 2) reinterpret_cast<uint16_t*>(p)[e] = (uint16_t)v;
        else reinterpret_cast<uint32_t*>(p)[e] = v;
      }
    }
  }
}

// Sum of squares of one chunk (Phase A, in-lane part). With DOT, bf16 rows
// use the gfx950 two-way bf16 dot product with a float32 accumulator, two
// squares per instruction straight from the packed words (products exact,
// denormal products kept), and FP8 rows first widen each pair of E4M3 values
// exactly to a bf16 pair for the same dot product. Without DOT (headwise
// kernels that widen the chunk to float32 for the scaling anyway and keep it)
// and for fp32 rows: a chain of fused multiply-adds in element order.
template <class IO, bool DOT>
__device__ __forceinline__ float chunk_sumsq(const Chunk& c) {
  float s = 0.0f;
  if constexpr (IO::kDtype == kDtypeBF16 && DOT) {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const bf16x2_t w = __builtin_bit_cast(bf16x2_t, c.w[p]);
      s = __builtin_amdgcn_fdot2_f32_bf16(w, w, s, false);
    }
  } else if constexpr (IO::kDtype == kDtypeFP8 && DOT) {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const bf16x2_t lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c.w[p], 1.0f, false);
      const bf16x2_t hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c.w[p], 1.0f, true);
      s = __builtin_amdgcn_fdot2_f32_bf16(lo, lo, s, false);
      s = __builtin_amdgcn_fdot2_f32_bf16(hi, hi, s, false);
    }
  } else {
    float v[IO::kVW];
    decode<IO>(c, v);
#pragma unroll
    for (int e = 0; e < IO::kVW; ++e) s = __builtin_fmaf(v[e], v[e], s);
  }
  return s;
}

// The layerwise row kernels sum bf16 and FP8 rows by dot products in every
// mode and for every slot count. The fused call and partial_stats must add
// the same values in the same order, or the split path (partial_stats, then
// apply_with_stats) would not reproduce the fused call bit for bit: a chain
// of fused multiply-adds rounds after every square, the dot product after
// every pair, and the two differ in the last bit of about 1% of bf16 chunk
// sums (and of FP8 chunks that mix large and small magnitudes).
template <class IO>
constexpr bool row_sums_by_dot() {
  return IO::kBytes < 4;
}

// The headwise kernels have no split path to agree with: packed rows held in
// up to 2 (bf16) or 4 (FP8) slots stay widened to float32 from the sums to the
// scaling, so their sums reuse that widening (measured faster there); above
// that the rows are widened again for the scaling and the dot products save
// the work.
template <class IO, int V>
constexpr bool head_sums_by_dot() {
  return IO::kBytes < 4 && V > (IO::kBytes == 2 ? 2 : 4);
}

// Phase B and the final scaling of FP8 rows in up to 4 slots: y = (x * gamma)
// * r[i], one rounding to E4M3, stores of the valid chunks (slot i goes to the
// Q or the K row). The saturating conversion costs four operations per
// element, so each chunk is converted without it and stored at once, four
// results at a time (no chunk's float32 results outlive its conversion),
// while the lane tracks its largest magnitude; only if some lane of the wave
// saw a result beyond 448 or a NaN does the wave convert its chunks again,
// saturated, and store them over the first results (a lane's two stores to
// one address land in program order). `gamma_at(i, e)` is element e of slot
// i's gamma as float32: widened from the packed bf16 words where it is used,
// or read from registers that hold it widened across tokens.
template <class IO, int V, bool ALIGNED, class GammaAt>
__device__ __forceinline__ void scale_store_fp8(const Chunk (&xv)[V], GammaAt gamma_at, const float (&r)[V],
                                                const bool (&isq)[V], const int (&col)[V], const int (&cnt)[V],
                                                char* yq_row, char* yk_row, bool active) {
  constexpr int VW = IO::kVW;
  float big = 0.0f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    Chunk out;
#pragma unroll
    for (int p = 0; p < 4; ++p) {  // elements 4p .. 4p+3: one word of x
      const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8(xv[i].w[p], false);
      const f32x2_t hi = __builtin_amdgcn_cvt_pk_f32_fp8(xv[i].w[p], true);
      const float y0 = (lo[0] * gamma_at(i, 4 * p)) * r[i];
      const float y1 = (lo[1] * gamma_at(i, 4 * p + 1)) * r[i];
      const float y2 = (hi[0] * gamma_at(i, 4 * p + 2)) * r[i];
      const float y3 = (hi[1] * gamma_at(i, 4 * p + 3)) * r[i];
      float m = __builtin_elementwise_maximum(__builtin_elementwise_maximum(big, __builtin_fabsf(y0)),
                                              __builtin_fabsf(y1));
      m = __builtin_elementwise_maximum(__builtin_elementwise_maximum(m, __builtin_fabsf(y2)), __builtin_fabsf(y3));
      big = cnt[i] > 0 ? m : big;  // idle slots left out
      out.w[p] = pack_fp8_word(y0, y1, y2, y3);
      // The word is formed here, not sunk into the store's branch (which
      // would keep all of the chunk's float32 results live until then).
      asm volatile("" : "+v"(out.w[p]));
      __builtin_amdgcn_sched_barrier(0);
    }
    if (active && cnt[i] > 0) store_chunk<IO, ALIGNED>(isq[i] ? yq_row : yk_row, col[i], cnt[i], out);
  }
  // A NaN (from gamma, say) sends the wave through the saturating path too,
  // which keeps NaN and clamps the rest.
  if (__builtin_amdgcn_ballot_w64(active && !(big <= 448.0f)) != 0) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float xf[VW], y[VW];
      decode<IO>(xv[i], xf);
#pragma unroll
      for (int e = 0; e < VW; ++e) y[e] = sat_e4m3((xf[e] * gamma_at(i, e)) * r[i]);
      Chunk out;
      pack<IO>(out, y);
      if (active && cnt[i] > 0) store_chunk<IO, ALIGNED>(isq[i] ? yq_row : yk_row, col[i], cnt[i], out);
    }
  }
}

// Phase B and the final scaling for this lane's chunks of one token:
// y = (x * gamma) * r[i], one rounding to the I/O type, stores of the valid
// chunks (slot i goes to the Q or the K row); FP8 rows in up to 4 slots take
// scale_store_fp8.
template <class IO, int V, bool ALIGNED>
__device__ __forceinline__ void scale_store(const Chunk (&xv)[V], const GChunk<IO> (&g)[V], const float (&r)[V],
                                            const bool (&isq)[V], const int (&col)[V], const int (&cnt)[V],
                                            char* yq_row, char* yk_row, bool active) {
  constexpr int VW = IO::kVW;
  if constexpr (IO::kDtype == kDtypeFP8 && V <= 4) {
    // element e of a chunk's gamma: the low or high bf16 half of word e / 2
    const auto gamma_at = [&](int i, int e) { return (e & 1) ? bf16_hi(g[i].w[e >> 1]) : bf16_lo(g[i].w[e >> 1]); };
    scale_store_fp8<IO, V, ALIGNED>(xv, gamma_at, r, isq, col, cnt, yq_row, yk_row, active);
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      if (active && cnt[i] > 0) {
        float xf[VW], gf[VW], y[VW];
        decode<IO>(xv[i], xf);
        decode_gamma<IO>(g[i], gf);
#pragma unroll
        for (int e = 0; e < VW; ++e) {
          y[e] = (xf[e] * gf[e]) * r[i];
          if (IO::kDtype == kDtypeFP8) y[e] = sat_e4m3(y[e]);  // many slots: clamp unconditionally
        }
        Chunk out;
        pack<IO>(out, y);
        store_chunk<IO, ALIGNED>(isq[i] ? yq_row : yk_row, col[i], cnt[i], out);
      }
    }
  }
}

// RMS factor of Eq. 1 for a global squared sum `ss`, full width H given as
// inv_div = 1/H (rounded once on the host): r = rsq(fma(ss, 1/H, eps)) with
// the hardware reciprocal square root (1 ulp). Where m = ss/H + eps falls
// below the float32 normal range, a subnormal m would keep too few bits, so
// m is formed again from ss * 2^64 and eps * 2^64 (both exact there) and r is
// scaled back by 2^32: one rounding in the normal range, as everywhere else.
// 0 gives +inf and +inf gives 0, as the formula does.
__device__ __forceinline__ float rms_factor(float ss, float inv_div, float eps) {
  float m = __builtin_fmaf(ss, inv_div, eps);
  const bool tiny = m < 1.17549435e-38f;  // false for NaN
  if (tiny) m = __builtin_fmaf(ss * 0x1p64f, inv_div, eps * 0x1p64f);
  const float r = __builtin_amdgcn_rsqf(m);
  return tiny ? r * 0x1p32f : r;
}

// Register-pressure guard: empty asm statements that claim to rewrite the
// words of `c`. Values the compiler widened from them earlier (bf16 or fp8 ->
// float32) can then not be kept alive across this point and are widened
// again where they are used, so packed data stays packed in registers.
// 16 bytes at a global-memory address held as an integer (a global load, not
// a flat one).
__device__ __forceinline__ Chunk load_global16(uint64_t addr) {
  typedef const u32x4_t __attribute__((address_space(1)))* gptr;
  const u32x4_t v = __builtin_nontemporal_load(reinterpret_cast<gptr>(addr));
  Chunk c;
  c.w[0] = v.x;
  c.w[1] = v.y;
  c.w[2] = v.z;
  c.w[3] = v.w;
  return c;
}

__device__ __forceinline__ uint32_t over(uint32_t n, const Divisor& d) {   // n / d
  return (uint32_t)((uint64_t)n * d.mul >> (31 + d.shift));
}

// One element that no kernel of the launch writes, at a wave-uniform address:
// through the constant address space the compiler uses a scalar load. As a
// vector load (what it emits where it cannot rule out a store to the same
// place) its use would wait for every row load issued before it.
template <class T>
__device__ __forceinline__ T load_uniform(const T* p) {
  typedef const T __attribute__((address_space(4)))* cptr;
  return *reinterpret_cast<cptr>(reinterpret_cast<uintptr_t>(p));
}

// A block-uniform 64-bit value, held in scalar registers: lanes that select
// between two such values then need no vector arithmetic to form them.
__device__ __forceinline__ uint64_t uniform64(uint64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)v);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(v >> 32));
  return ((uint64_t)hi << 32) | lo;
}

template <int W>
__device__ __forceinline__ void keep_packed(Words<W>& c) {
#pragma unroll
  for (int q = 0; q < W; ++q) asm volatile("" : "+v"(c.w[q]));
}

// Sum over aligned groups of `group` lanes (a power of two, 1..64); every
// lane of a group ends with the same value. Inside a 16-lane row the steps
// are DPP moves fused into the adds (quad permutes, then the half-row and
// row mirrors, which pair lanes of the two halves once each half is
// uniform). The 16- and 32-lane steps cross rows with gfx950's permlane
// swaps (measured faster than the LDS crossbar for every I/O type):
// swapping the odd rows (or the upper half) of one copy with the even rows
// (lower half) of another leaves row pairs (halves) side by side in the two
// results, so one add gives every lane the pair's sum. Each step adds two
// lanes' values, a + b on one and b + a (or a + b) on the other, so all
// lanes of a group hold bitwise the same sum.
template <int CTRL>
__device__ __forceinline__ float dpp_move(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, false));
}

__device__ __forceinline__ float swap_add16(float v) {  // lanes i ^ 16
  const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(p[0]) + __uint_as_float(p[1]);
}

__device__ __forceinline__ float swap_add32(float v) {  // lanes i ^ 32
  const auto p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(p[0]) + __uint_as_float(p[1]);
}

template <int GROUP>
__device__ __forceinline__ float group_sum_of(float v) {
  if (GROUP > 1) v += dpp_move<0xB1>(v);    // lanes i ^ 1   (quad_perm 1,0,3,2)
  if (GROUP > 2) v += dpp_move<0x4E>(v);    // lanes i ^ 2   (quad_perm 2,3,0,1)
  if (GROUP > 4) v += dpp_move<0x141>(v);   // lanes 7 - i within 8 (row_half_mirror)
  if (GROUP > 8) v += dpp_move<0x140>(v);   // lanes 15 - i within 16 (row_mirror)
  if (GROUP > 16) v = swap_add16(v);
  if (GROUP > 32) v = swap_add32(v);
  return v;
}

// The group width is uniform over the launch: one test picks the straight
// sequence of steps (a test per step compiled to a branch and a
// materialised condition each, for every token).
__device__ __forceinline__ float group_sum(float v, int group) {
  if (group == 64) return group_sum_of<64>(v);  // most launches: tested first
  switch (group) {
    case 32: return group_sum_of<32>(v);
    case 16: return group_sum_of<16>(v);
    case 8: return group_sum_of<8>(v);
    case 4: return group_sum_of<4>(v);
    case 2: return group_sum_of<2>(v);
    default: return v;
  }
}

// The Q and K sums of a group together, each bitwise equal to group_sum_of
// on it alone. Groups of 32 and 64 lanes take the in-row steps for each sum
// separately, then share the steps across rows: one permlane16 swap of the
// (Q, K) pair leaves rows of Q0|K0|Q2|K2 in one register and Q1|K1|Q3|K3 in
// the other, so a single add forms the row-pair sums of both (Q in the even
// rows, K in the odd ones, each added as the separate step adds it); a
// permlane32 swap and add then forms the 64-lane sums the same way, and a
// last permlane16 swap hands every lane both sums. Five to six instructions
// instead of ten to twelve.
template <int GROUP>
__device__ __forceinline__ void group_sum_qk_of(float& q, float& k) {
  if constexpr (GROUP < 32) {
    q = group_sum_of<GROUP>(q);
    k = group_sum_of<GROUP>(k);
  } else {
    q = group_sum_of<16>(q);
    k = group_sum_of<16>(k);
    const auto rows = __builtin_amdgcn_permlane16_swap(__float_as_uint(q), __float_as_uint(k), false, false);
    float w = __uint_as_float(rows[0]) + __uint_as_float(rows[1]);  // Q01 | K01 | Q23 | K23
    if constexpr (GROUP > 32) {
      const auto halves = __builtin_amdgcn_permlane32_swap(__float_as_uint(w), __float_as_uint(w), false, false);
      w = __uint_as_float(halves[0]) + __uint_as_float(halves[1]);  // Q | K | Q | K
    }
    const auto both = __builtin_amdgcn_permlane16_swap(__float_as_uint(w), __float_as_uint(w), false, false);
    q = __uint_as_float(both[0]);
    k = __uint_as_float(both[1]);
  }
}

__device__ __forceinline__ void group_sum_qk(float& q, float& k, int group) {
  if (group == 64) return group_sum_qk_of<64>(q, k);
  switch (group) {
    case 32: return group_sum_qk_of<32>(q, k);
    case 16: return group_sum_qk_of<16>(q, k);
    case 8: return group_sum_qk_of<8>(q, k);
    case 4: return group_sum_qk_of<4>(q, k);
    case 2: return group_sum_qk_of<2>(q, k);
    default: return;
  }
}

__device__ __forceinline__ float lane_read(float v, int lane) {
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), lane));
}

}  // namespace
}  // namespace qkn

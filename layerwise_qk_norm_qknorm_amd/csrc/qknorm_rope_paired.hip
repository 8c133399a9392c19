// The kernels of qknorm_rope.hip for the heads its layout does not take: head
// widths or rotations whose 16-byte chunks are no power of two, odd sizes and
// unaligned rows.
//
// A lane owns pairs of pieces (A, B) of one head, each 16 or 8 bytes or one
// element wide: for the half-split rotation A lies in the first half and B in
// the second, at the same offset, so both members of every pair are in one
// lane. The head's sum of squares is a butterfly over its lanes. One pass of a
// wave over 64 / lanes heads is a slot; slots never mix Q, K and V, so all
// that depends on the side is scalar.
//
// 8192 tokens x 48 bf16 heads: of 80 columns 40.8 us (3.2 TB/s: 5 of 8 lanes
// hold pairs), of 96 columns 43.1 (3.6 TB/s); their gradients 49.7 and 59.6 (3.9
// TB/s); 40 + 8 + 8 heads of 96 into a 4-bit cache 71.3 (2.3 TB/s: every key in
// float64).

#include "qknorm_rope_device.hpp"

#include <string>
#include <type_traits>

namespace qkn {
namespace {

// Where a lane's pairs lie in a head. Rotated pairs come first: half-split,
// piece p of each half; interleaved (and the columns past `rot`), two
// neighbouring pieces. The cos and sin of pair p start at p * VW for both.
template <int VW, int NP, bool INTER>
struct Place {
  int a[NP], b[NP];
  int tab[NP];        // offset of the pair's cos (0 where not rotated)
  bool turn[NP];      // rotated
  bool has_a[NP], has_b[NP];
  __device__ __forceinline__ Place(int lane_in_head, int lanes, int pairs, int rot_pairs, int rot, int head_dim) {
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      const int p = lane_in_head + k * lanes;
      turn[k] = p < rot_pairs;
      a[k] = INTER || !turn[k] ? 2 * p * VW : p * VW;
      b[k] = INTER || !turn[k] ? a[k] + VW : (rot >> 1) + p * VW;
      tab[k] = turn[k] ? p * VW : 0;
      has_a[k] = p < pairs;
      has_b[k] = has_a[k] && (VW > 1 || b[k] < head_dim);
      a[k] = has_a[k] ? a[k] : 0;   // idle: reads the head's first piece
      b[k] = has_b[k] ? b[k] : 0;
    }
  }
};

// Zeroes the pieces that a head does not have (a lane without a pair, the odd
// column of an odd head), so that they add nothing to the head's sums. Only
// where a head leaves lanes idle.
template <int PB, int VW, int NP, bool INTER>
__device__ __forceinline__ void drop_idle(Piece<PB> (&a)[NP], Piece<PB> (&b)[NP], const Place<VW, NP, INTER>& at) {
#pragma unroll
  for (int k = 0; k < NP; ++k)
#pragma unroll
    for (int q = 0; q < (PB >= 4 ? PB / 4 : 1); ++q) {
      a[k].w[q] = at.has_a[k] ? a[k].w[q] : 0u;
      b[k].w[q] = at.has_b[k] ? b[k].w[q] : 0u;
    }
}

// cos and sin of the lane's pairs at one position. A position outside the
// table gives NaN, which reaches every rotated column of the token.
template <int VW, int NP, bool INTER, bool AXES>
struct Angles {
  float c[NP][VW], s[NP][VW];
  // AXES: positions on several axes, gathered by the wave and read from LDS
  static constexpr int kRounds = AXES ? kRopeMaxHead / 2 / 64 : 1;
  static constexpr int kLds = AXES ? 2 * 64 * kRounds : 1;   // floats a wave
  AxisAngles own;
  template <class Args>
  __device__ __forceinline__ void load(const Args& a, int64_t t, const Place<VW, NP, INTER>& at, uint32_t axes) {
    if constexpr (AXES) {
      AxisAngles::Positions pos;
      pos.load(a, t);
      own.load(a, pos, axes);
    } else
      load(a.cos_sin, a.ld_table, a.n_positions, load_uniform(a.positions + t), a.rot >> 1, at);
  }
  template <class Args>
  __device__ __forceinline__ void settle(const Args& a, int64_t t, float* lds, const Place<VW, NP, INTER>& at) {
    if constexpr (AXES) {
      own.template put<kRounds>(a, t, lds);
#pragma unroll
      for (int k = 0; k < NP; ++k)
#pragma unroll
        for (int e = 0; e < VW; ++e) {
          c[k][e] = lds[at.tab[k] + e];
          s[k][e] = lds[kSinAt(kRounds) + at.tab[k] + e];
        }
    }
  }
  __device__ __forceinline__ void load(const float* table, int64_t ld, int64_t n, int64_t pos, int half,
                                       const Place<VW, NP, INTER>& at) {
    const bool in = pos >= 0 && pos < n;
    const float* row = table + (in ? pos : 0) * ld;
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      load_bytes<VW * 4, false>(reinterpret_cast<const char*>(row + at.tab[k]), reinterpret_cast<uint32_t*>(c[k]));
      load_bytes<VW * 4, false>(reinterpret_cast<const char*>(row + half + at.tab[k]),
                                reinterpret_cast<uint32_t*>(s[k]));
    }
    if (!in) {
      keep_branch();
#pragma unroll
      for (int k = 0; k < NP; ++k)
#pragma unroll
        for (int e = 0; e < VW; ++e) c[k][e] = s[k][e] = __builtin_nanf("");
    }
  }
};

// Rotates one lane's pieces of a head (BACK: by the opposite angle, the
// transposed map that gradients take).
template <class F, int VW, bool INTER, bool BACK>
__device__ __forceinline__ void rotate(F (&a)[VW], F (&b)[VW], const float (&c)[VW], const float (&s)[VW]) {
  if constexpr (INTER && VW > 1) {
#pragma unroll
    for (int i = 0; i < VW / 2; ++i) {
      const F ca = c[i], sa = BACK ? -s[i] : s[i], cb = c[VW / 2 + i], sb = BACK ? -s[VW / 2 + i] : s[VW / 2 + i];
      const F a0 = a[2 * i], a1 = a[2 * i + 1], b0 = b[2 * i], b1 = b[2 * i + 1];
      a[2 * i] = a0 * ca - a1 * sa;
      a[2 * i + 1] = a1 * ca + a0 * sa;
      b[2 * i] = b0 * cb - b1 * sb;
      b[2 * i + 1] = b1 * cb + b0 * sb;
    }
  } else {
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      const F ce = c[e], se = BACK ? -s[e] : s[e];
      const F a0 = a[e], b0 = b[e];
      a[e] = a0 * ce - b0 * se;
      b[e] = b0 * ce + a0 * se;
    }
  }
}

// Most float32 values of one slot's heads (one wave's exchange buffer).
constexpr int kSlotValues = 1024;

// One wave's slot of K or V values, float32 in `val` ([heads][head_dim]), into
// the codes of a quantised cache. Four lanes hold a block, eight channels each.
template <class IO, class MX>
__device__ __forceinline__ void quantize_slot(const float* val, const RopeArgs& a, int lane, int heads_here,
                                              int head0, char* codes, char* scales, char* y_row) {
  const int per_head = a.head_dim >> 3;   // eight-channel pieces
  const int total = heads_here * per_head;
#pragma unroll 1
  for (int i0 = 0; i0 < total; i0 += 64) {
    const int i = i0 + lane;
    const bool on = i < total;            // the same for the four lanes of a block
    const int h = on ? i / per_head : 0;
    const int c = on ? (i - h * per_head) * 8 : 0;
    float f[8];
#pragma unroll
    for (int q = 0; q < 8; q += 4) {
      const f32x4_t v = *reinterpret_cast<const f32x4_t*>(val + h * a.head_dim + c + q);
      f[q] = v[0];
      f[q + 1] = v[1];
      f[q + 2] = v[2];
      f[q + 3] = v[3];
    }
    uint32_t m = 0;                       // largest magnitude, as ordered bits: NaN above infinity
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(f[e]) & 0x7FFFFFFFu);
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, false));
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, false));
    const int byte = scale_byte<MX>(m);
    const float inv = over_scale(byte);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] = byte == 0xFF ? 0.0f : MX::saturated(f[e] * inv);
    const Codes<MX, 8> w = codes_of<MX, 8>(f);
    if (on) {
      store_bytes<MX::kBits>(codes + (int64_t)(head0 + h) * a.head_stride + c * MX::kBits / 8, w.w);
      if ((lane & 3) == 0) scales[(int64_t)(head0 + h) * a.scale_head_stride + (c >> 5)] = (char)byte;
      if (y_row) {   // what the cache now holds, in the row type (exact)
        float y[8];
        code_values<MX, 8>(w, byte, y);
        uint32_t o[IO::kBytes * 2];
        narrow<IO, 8>(y, o);
        char* p = y_row + ((int64_t)(head0 + h) * a.head_dim + c) * IO::kBytes;
        if (a.y_wide) {
#pragma unroll
          for (int q = 0; q < IO::kBytes / 2; ++q) store_bytes<16>(p + 16 * q, o + 4 * q);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const uint32_t one = IO::kBytes == 4 ? o[e] : o[e >> 1] >> (16 * (e & 1));
            store_bytes<IO::kBytes>(p + e * IO::kBytes, &one);
          }
        }
      }
    }
  }
}

// The forward pass (MODE ROPE_FORWARD: Q and K rows to y) and the append
// calls (Q to y, K and V into the cache). Block: `waves` waves per token,
// each with S slots of it, `tokens` tokens; grid.y covers the slots past a
// block's waves. All loads of a wave's slots are issued before the first is
// used.
template <class IO, int PB, int NP, int S, bool INTER, int MODE, bool AXES>
__global__ void __launch_bounds__(64 * kRopeMaxWaves) qknorm_rope_paired(const std::conditional_t<AXES, RopeAxesArgs, RopeArgs> a) {
  constexpr bool CODES = MODE == ROPE_APPEND_MXFP4 || MODE == ROPE_APPEND_MXFP8;
  using MX = std::conditional_t<MODE == ROPE_APPEND_MXFP8, Mx8, Mx4>;
  constexpr int VW = PB / IO::kBytes;
  constexpr int GB = VW * IO::kGBytes;
  __shared__ __align__(16) float exchange[CODES ? kRopeMaxWaves * kSlotValues : 4];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tok = (int)((uint32_t)wave * a.waves_inv >> 16);           // wave / waves
  const int slot0 = (blockIdx.y * a.waves + (wave - tok * a.waves)) * S;
  if (slot0 >= a.n_slots) return;
  const int L = 1 << a.log2_lanes;
  const int hl = lane >> a.log2_lanes;
  const int hw = 64 >> a.log2_lanes;
  const Place<VW, NP, INTER> at(lane & (L - 1), L, a.pairs, a.rot_pairs, a.rot, a.head_dim);

  using Turns = Angles<VW, NP, INTER, AXES>;
  __shared__ __align__(16) float angles[kRopeMaxWaves * Turns::kLds];
  float* const lds = angles + wave * Turns::kLds;
  const uint32_t axes = lane_axes(a);

  // What the wave's slots hold, the same for all its tokens: the side (Q, K or
  // V), the lane's byte offset in its rows, and gamma.
  int side[S];
  uint32_t oa[S][NP], ob[S][NP];
  Piece<GB> ga[S][NP], gb[S][NP];
#pragma unroll
  for (int i = 0; i < S; ++i) {
    const int s = min(slot0 + i, a.n_slots - 1);
    side[i] = s < a.first[1] ? 0 : MODE != ROPE_FORWARD && s >= a.first[2] ? 2 : 1;
    const RopeSide& o = a.side[side[i]];
    const int head = (s - a.first[side[i]]) * hw + hl;
    const int hc = head < o.heads ? head : 0;    // idle lanes read the first head
    const char* g = static_cast<const char*>(o.gamma);
    if (g) g += hc * a.gstride * IO::kGBytes;
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      oa[i][k] = (uint32_t)(hc * a.head_dim + at.a[k]) * IO::kBytes;
      ob[i][k] = (uint32_t)(hc * a.head_dim + at.b[k]) * IO::kBytes;
      if (g) {
        load_bytes<GB, false>(g + at.a[k] * IO::kGBytes, ga[i][k].w);
        load_bytes<GB, false>(g + at.b[k] * IO::kGBytes, gb[i][k].w);
      }
    }
  }

  struct In {   // one token
    Piece<PB> xa[S][NP], xb[S][NP];
    Turns turn;
    int64_t place;
  };
  const auto load = [&](In& in, int64_t t) {
    if constexpr (MODE != ROPE_FORWARD) in.place = load_uniform(a.slots + t);
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const RopeSide& o = a.side[side[i]];
      const char* row = static_cast<const char*>(o.x) + t * o.ldx * IO::kBytes;
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        load_bytes<PB, true>(row + oa[i][k], in.xa[i][k].w);
        load_bytes<PB, true>(row + ob[i][k], in.xb[i][k].w);
      }
    }
    if (a.rot_pairs) in.turn.load(a, t, at, axes);
  };

  const auto work = [&](In& in, int64_t t) {
    if (MODE != ROPE_FORWARD && (in.place < 0 || in.place >= a.n_tokens_held)) return;   // a row that holds no token
    if (a.rot_pairs) in.turn.settle(a, t, lds, at);
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const int s = slot0 + i;
      if (s >= a.n_slots) break;
      const int c = side[i];
      const RopeSide& o = a.side[c];
      const int head0 = (s - a.first[c]) * hw;
      const bool on = head0 + hl < o.heads;
      if (a.idle) {
        keep_branch();
        drop_idle<PB, VW, NP, INTER>(in.xa[i], in.xb[i], at);
      }
      float fa[NP][VW], fb[NP][VW];
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        widen<IO, VW>(in.xa[i][k].w, fa[k]);
        widen<IO, VW>(in.xb[i][k].w, fb[k]);
      }
      const bool exact = CODES && c == 1;
      if (exact) {
        // Keys bound for codes: formed in float64 (vector float64 runs
        // at the float32 rate here), so that every code is the one exact
        // arithmetic gives and does not hang on the order of a sum.
        double r = 1.0;
        if (o.gamma) {
          double ss = 0.0;
#pragma unroll
          for (int k = 0; k < NP; ++k)
#pragma unroll
            for (int e = 0; e < VW; ++e) {
              const double va = fa[k][e], vb = fb[k][e];
              ss += va * va + vb * vb;
            }
          ss = group_sum_d(ss, L);
          r = 1.0 / __builtin_sqrt(ss / a.head_dim + (double)a.eps);
        }
#pragma unroll
        for (int k = 0; k < NP; ++k) {
          double da[VW], db[VW];
          float gfa[VW], gfb[VW];
          if (o.gamma) {
            widen_gamma<IO, VW>(ga[i][k].w, gfa);
            widen_gamma<IO, VW>(gb[i][k].w, gfb);
          }
#pragma unroll
          for (int e = 0; e < VW; ++e) {
            da[e] = o.gamma ? (double)fa[k][e] * gfa[e] * r : (double)fa[k][e];
            db[e] = o.gamma ? (double)fb[k][e] * gfb[e] * r : (double)fb[k][e];
          }
          if (at.turn[k]) rotate<double, VW, INTER, false>(da, db, in.turn.c[k], in.turn.s[k]);
#pragma unroll
          for (int e = 0; e < VW; ++e) {
            fa[k][e] = round_to_odd(da[e]);
            fb[k][e] = round_to_odd(db[e]);
          }
        }
      } else if (c != 2) {
        if (o.gamma) {
          float ss = 0.0f;
#pragma unroll
          for (int k = 0; k < NP; ++k)
#pragma unroll
            for (int e = 0; e < VW; ++e) {
              ss = __builtin_fmaf(fa[k][e], fa[k][e], ss);
              ss = __builtin_fmaf(fb[k][e], fb[k][e], ss);
            }
          ss = group_sum(ss, L);
          const float r = rms_factor(ss, a.inv_div, a.eps);
#pragma unroll
          for (int k = 0; k < NP; ++k) {
            float gfa[VW], gfb[VW];
            widen_gamma<IO, VW>(ga[i][k].w, gfa);
            widen_gamma<IO, VW>(gb[i][k].w, gfb);
#pragma unroll
            for (int e = 0; e < VW; ++e) {
              fa[k][e] = (fa[k][e] * gfa[e]) * r;
              fb[k][e] = (fb[k][e] * gfb[e]) * r;
            }
          }
        }
#pragma unroll
        for (int k = 0; k < NP; ++k)
          if (at.turn[k]) rotate<float, VW, INTER, false>(fa[k], fb[k], in.turn.c[k], in.turn.s[k]);
      }

      char* y_row = o.y ? static_cast<char*>(o.y) + t * o.ldy * IO::kBytes : nullptr;
      if (CODES && c != 0) {
        float* ex = exchange + wave * kSlotValues;
#pragma unroll
        for (int k = 0; k < NP; ++k)
#pragma unroll
          for (int e = 0; e < VW; ++e) {
            if (at.has_a[k]) ex[hl * a.head_dim + at.a[k] + e] = fa[k][e];
            if (at.has_b[k]) ex[hl * a.head_dim + at.b[k] + e] = fb[k][e];
          }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        const int64_t page = in.place >> a.log2_page, off = in.place & (((int64_t)1 << a.log2_page) - 1);
        char* codes = a.cache[c - 1] + page * a.page_stride + off * a.token_stride;
        char* scales = a.scales[c - 1] + page * a.scale_page_stride + off * (a.head_dim >> 5);
        quantize_slot<IO, MX>(ex, a, lane, min(hw, o.heads - head0), head0, codes, scales, y_row);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        continue;
      }
      if (!on) continue;
#pragma unroll
      for (int k = 0; k < NP; ++k) {
        Piece<PB> ya, yb;
        narrow<IO, VW>(fa[k], ya.w);
        narrow<IO, VW>(fb[k], yb.w);
        if (MODE == ROPE_APPEND_ROWS && c != 0) {
          const int64_t page = in.place >> a.log2_page, off = in.place & (((int64_t)1 << a.log2_page) - 1);
          char* p = a.cache[c - 1] + page * a.page_stride + off * a.token_stride + (int64_t)(head0 + hl) * a.head_stride;
          if (at.has_a[k]) store_bytes<PB>(p + at.a[k] * IO::kBytes, ya.w);
          if (at.has_b[k]) store_bytes<PB>(p + at.b[k] * IO::kBytes, yb.w);
        }
        if (y_row) {
          if (at.has_a[k]) store_bytes<PB>(y_row + oa[i][k], ya.w);
          if (at.has_b[k]) store_bytes<PB>(y_row + ob[i][k], yb.w);
        }
      }
    }
  };

  const int64_t step = (int64_t)gridDim.x * a.tokens;
  each_token<In>((int64_t)blockIdx.x * a.tokens + tok, step, a.T, load, work);
}

// Gradients. With g the incoming gradient turned back by the rotation, xr =
// x * r and gg = g * gamma: dgamma_j = sum over tokens (and heads sharing
// gamma) of g_j xr_j, and dx = r (gg - xr mean(gg xr)). x and dy are read
// once, dx written once; everything between stays in registers. A wave keeps
// one slot of heads for all its tokens, so its share of dgamma stays in
// registers too and leaves as one partial row per block (its waves added in
// LDS in a fixed order); qknorm_rope_grad_sum adds the rows in a fixed
// order, so the gradients do not change from run to run. The next token's
// loads are issued before the current one is worked on.
template <class IO, int PB, int NP, bool INTER, bool AXES>
__global__ void __launch_bounds__(64 * kGradWaves, 3) qknorm_rope_paired_grad(const std::conditional_t<AXES, RopeGradAxesArgs, RopeGradArgs> a) {
  constexpr int VW = PB / IO::kBytes;
  constexpr int GB = VW * IO::kGBytes;
  constexpr int E = 2 * NP * VW;
  __shared__ float red[kGradWaves * 64 * E];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int s = blockIdx.y;
  const int c = s < a.first[1] ? 0 : 1;
  const RopeGradSide& o = a.side[c];
  const int L = 1 << a.log2_lanes;
  const int hl = lane >> a.log2_lanes;
  const int hw = 64 >> a.log2_lanes;
  const int head = (s - a.first[c]) * hw + hl;
  const bool on = head < o.heads;
  const int hc = on ? head : 0;
  const Place<VW, NP, INTER> at(lane & (L - 1), L, a.pairs, a.rot_pairs, a.rot, a.head_dim);

  using Turns = Angles<VW, NP, INTER, AXES>;
  __shared__ __align__(16) float angles[kGradWaves * Turns::kLds];
  float* const lds = angles + wave * Turns::kLds;
  const uint32_t axes = lane_axes(a);

  float gfa[NP][VW], gfb[NP][VW];
  float sa[NP][VW], sb[NP][VW];
  uint32_t oa[NP], ob[NP];
  {
    const char* g = static_cast<const char*>(o.gamma) + hc * a.gstride * IO::kGBytes;
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      Piece<GB> p;
      load_bytes<GB, false>(g + at.a[k] * IO::kGBytes, p.w);
      widen_gamma<IO, VW>(p.w, gfa[k]);
      load_bytes<GB, false>(g + at.b[k] * IO::kGBytes, p.w);
      widen_gamma<IO, VW>(p.w, gfb[k]);
#pragma unroll
      for (int e = 0; e < VW; ++e) sa[k][e] = sb[k][e] = 0.0f;
      oa[k] = (uint32_t)(hc * a.head_dim + at.a[k]) * IO::kBytes;
      ob[k] = (uint32_t)(hc * a.head_dim + at.b[k]) * IO::kBytes;
    }
  }
  const char* x = static_cast<const char*>(o.x);
  const char* dy = static_cast<const char*>(o.dy);
  char* dx = static_cast<char*>(o.dx);

  struct In {
    Piece<PB> xa[NP], xb[NP], ya[NP], yb[NP];
    Turns turn;
  };
  const auto load = [&](In& in, int64_t t) {
    const char* xr = x + t * o.ldx * IO::kBytes;
    const char* yr = dy + t * o.lddy * IO::kBytes;
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      load_bytes<PB, true>(xr + oa[k], in.xa[k].w);
      load_bytes<PB, true>(xr + ob[k], in.xb[k].w);
      load_bytes<PB, true>(yr + oa[k], in.ya[k].w);
      load_bytes<PB, true>(yr + ob[k], in.yb[k].w);
    }
    if (a.rot_pairs) in.turn.load(a, t, at, axes);
  };
  const auto work = [&](In& in, int64_t t) {
    if (a.rot_pairs) in.turn.settle(a, t, lds, at);
    if (a.idle) {
      keep_branch();
      drop_idle<PB, VW, NP, INTER>(in.xa, in.xb, at);
    }
    float xa[NP][VW], xb[NP][VW], ya[NP][VW], yb[NP][VW], pa[NP][VW], pb[NP][VW];
    float ss = 0.0f, dot = 0.0f;
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      widen<IO, VW>(in.xa[k].w, xa[k]);
      widen<IO, VW>(in.xb[k].w, xb[k]);
      widen<IO, VW>(in.ya[k].w, ya[k]);
      widen<IO, VW>(in.yb[k].w, yb[k]);
      if (at.turn[k]) rotate<float, VW, INTER, true>(ya[k], yb[k], in.turn.c[k], in.turn.s[k]);
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        ss = __builtin_fmaf(xa[k][e], xa[k][e], ss);
        ss = __builtin_fmaf(xb[k][e], xb[k][e], ss);
        pa[k][e] = ya[k][e] * gfa[k][e];
        pb[k][e] = yb[k][e] * gfb[k][e];
        dot = __builtin_fmaf(pa[k][e], xa[k][e], dot);
        dot = __builtin_fmaf(pb[k][e], xb[k][e], dot);
      }
    }
    group_sum_qk(ss, dot, L);
    const float r = rms_factor(ss, a.inv_div, a.eps);
    const float mean = (dot * r) * a.inv_div;
    char* row = dx + t * o.lddx * IO::kBytes;
#pragma unroll
    for (int k = 0; k < NP; ++k) {
      float da[VW], db[VW];
#pragma unroll
      for (int e = 0; e < VW; ++e) {
        const float ra = xa[k][e] * r, rb = xb[k][e] * r;
        sa[k][e] = __builtin_fmaf(ya[k][e], ra, sa[k][e]);
        sb[k][e] = __builtin_fmaf(yb[k][e], rb, sb[k][e]);
        da[e] = r * __builtin_fmaf(-ra, mean, pa[k][e]);
        db[e] = r * __builtin_fmaf(-rb, mean, pb[k][e]);
      }
      if (on) {
        Piece<PB> p;
        narrow<IO, VW>(da, p.w);
        if (at.has_a[k]) store_bytes<PB>(row + oa[k], p.w);
        narrow<IO, VW>(db, p.w);
        if (at.has_b[k]) store_bytes<PB>(row + ob[k], p.w);
      }
    }
  };

  each_token<In>((int64_t)blockIdx.x * kGradWaves + wave, (int64_t)a.workers * kGradWaves, a.T, load, work);

  if (!o.dgamma) return;
#pragma unroll
  for (int k = 0; k < NP; ++k)
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      red[(wave * E + k * 2 * VW + e) * 64 + lane] = sa[k][e];
      red[(wave * E + (k * 2 + 1) * VW + e) * 64 + lane] = sb[k][e];
    }
  __syncthreads();
  // Shared gamma: one row per (slot, worker), the slot's heads added too;
  // otherwise one row per (head, worker).
  const bool shared = a.gstride == 0;
  const int live = min(hw, o.heads - (s - a.first[c]) * hw);   // heads of this slot
  for (int i = threadIdx.x; i < E * 64; i += 64 * kGradWaves) {
    const int l = i & 63, e = i >> 6;
    const int lh = l >> a.log2_lanes;
    if (shared ? lh != 0 : lh >= live) continue;
    float sum = 0.0f;
    for (int h = 0; h < (shared ? live : 1); ++h)
      for (int w = 0; w < kGradWaves; ++w) sum += red[(w * E + e) * 64 + l + (h << a.log2_lanes)];
    // column of (lane, e): the lane's k-th pair, side A or B, element
    const int k = e / (2 * VW), side = (e / VW) & 1, el = e % VW;
    const int p = (l & (L - 1)) + k * L;
    const bool turned = p < a.rot_pairs;
    const int ca = INTER || !turned ? 2 * p * VW : p * VW;
    const int cb = INTER || !turned ? ca + VW : (a.rot >> 1) + p * VW;
    const int col = (side ? cb : ca) + el;
    if (p >= a.pairs || col >= a.head_dim) continue;
    const int global_head = (c ? a.side[0].heads : 0) + (s - a.first[c]) * hw + lh;
    const int64_t row = shared ? (int64_t)s * a.workers + blockIdx.x : (int64_t)global_head * a.workers + blockIdx.x;
    a.partial[row * a.head_dim + col] = sum;
  }
}

using RopeFn = const void*;      // kernels of two argument types
using GradFn = const void*;

template <class IO, bool INTER, int MODE, bool AXES>
RopeFn pick_rope(const RopePlan& p) {
  if (p.piece_bytes == 16) {
    switch (p.slots) {
      case 1: return reinterpret_cast<const void*>(qknorm_rope_paired<IO, 16, 1, 1, INTER, MODE, AXES>);
      case 3: return reinterpret_cast<const void*>(qknorm_rope_paired<IO, 16, 1, 3, INTER, MODE, AXES>);
    }
    return nullptr;
  }
  if (p.slots != 1) return nullptr;
  if (p.piece_bytes == 8) return reinterpret_cast<const void*>(qknorm_rope_paired<IO, 8, 1, 1, INTER, MODE, AXES>);
  if (p.np == 1) return reinterpret_cast<const void*>(qknorm_rope_paired<IO, IO::kBytes, 1, 1, INTER, MODE, AXES>);
  return reinterpret_cast<const void*>(qknorm_rope_paired<IO, IO::kBytes, 8, 1, INTER, MODE, AXES>);
}

template <class IO, bool INTER, bool AXES>
RopeFn pick_rope_mode(int mode, const RopePlan& p) {
  if (mode == ROPE_FORWARD) return pick_rope<IO, INTER, ROPE_FORWARD, AXES>(p);
  if constexpr (IO::kBytes > 1) {
    if (mode == ROPE_APPEND_ROWS) return pick_rope<IO, INTER, ROPE_APPEND_ROWS, AXES>(p);
    if (mode == ROPE_APPEND_MXFP8) return pick_rope<IO, INTER, ROPE_APPEND_MXFP8, AXES>(p);
    return pick_rope<IO, INTER, ROPE_APPEND_MXFP4, AXES>(p);
  }
  return nullptr;
}

template <class IO>
RopeFn pick_rope_turn(int mode, bool inter, bool axes, const RopePlan& p) {
  if (axes) return inter ? pick_rope_mode<IO, true, true>(mode, p) : pick_rope_mode<IO, false, true>(mode, p);
  return inter ? pick_rope_mode<IO, true, false>(mode, p) : pick_rope_mode<IO, false, false>(mode, p);
}

template <class IO, bool INTER, bool AXES>
GradFn pick_grad(const RopePlan& p) {
  if (p.piece_bytes == 16) return reinterpret_cast<const void*>(qknorm_rope_paired_grad<IO, 16, 1, INTER, AXES>);
  if (p.piece_bytes == 8) return reinterpret_cast<const void*>(qknorm_rope_paired_grad<IO, 8, 1, INTER, AXES>);
  if (p.np == 1) return reinterpret_cast<const void*>(qknorm_rope_paired_grad<IO, IO::kBytes, 1, INTER, AXES>);
  return reinterpret_cast<const void*>(qknorm_rope_paired_grad<IO, IO::kBytes, 8, INTER, AXES>);
}

template <class IO>
GradFn pick_grad_turn(bool inter, bool axes, const RopePlan& p) {
  if (axes) return inter ? pick_grad<IO, true, true>(p) : pick_grad<IO, false, true>(p);
  return inter ? pick_grad<IO, true, false>(p) : pick_grad<IO, false, false>(p);
}

}  // namespace

const void* rope_paired_kernel(int mode, int dtype, bool inter, bool axes, const RopePlan& p) {
  return dtype == kDtypeBF16  ? pick_rope_turn<BF16>(mode, inter, axes, p)
         : dtype == kDtypeF32 ? pick_rope_turn<F32>(mode, inter, axes, p)
                              : pick_rope_turn<FP8>(mode, inter, axes, p);
}

const void* rope_paired_grad_kernel(int dtype, bool inter, bool axes, const RopePlan& p) {
  return dtype == kDtypeBF16 ? pick_grad_turn<BF16>(inter, axes, p) : pick_grad_turn<F32>(inter, axes, p);
}

}  // namespace qkn

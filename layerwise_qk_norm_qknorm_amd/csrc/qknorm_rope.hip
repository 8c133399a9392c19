// HIP kernels for headwise QK-Norm with the position rotation in the same
// pass, its gradients, and appending keys and values to a paged cache, on
// gfx950 (CDNA4).
//
// Per head of d columns: z = x * gamma * r with r = 1/sqrt(sum x^2 / d + eps)
// (Eq. 1 per head; no gamma: z = x), then every pair (a, b) of the first
// `rot` columns becomes (a c - b s, b c + a s) with the cos and sin of its
// position's angle, read from a table.
//
// All of it streams: a few flops per byte, so the kernels are bound by HBM.
// Each element is read once and written once; what a lane needs of the table
// is loaded once per token and used for every head the wave holds.
//
// Work layout: a head of L 16-byte chunks, L a power of two (128 bf16 columns:
// 16), is held by L neighbouring lanes, one chunk each, so that every load and
// store of a wave covers 1 KiB in a row (64 / L heads: a slot). For the
// half-split rotation the other member of a lane's pairs is L/2 lanes away
// (rot/2 columns), a DPP move inside a 16-lane row and a permlane swap across
// rows. The first layout tried kept both members of a pair in one lane, which
// needs no exchange but reads a head in two 128-byte runs per instruction.
// 8192 tokens x 48 heads x 128 bf16 columns: half-split 39.0 -> 36.6 us (5.6
// TB/s; float32 71.5, 5.7 TB/s; FP8 35.7, bound by its conversions), interleaved 45 -> 36.6, no rotation 43 -> 36; gradients 79 -> 59.
// Positions on three axes add the gathering of the token's angles by each wave (351
// vector instructions a wave, 275 with one position): 38.7 us and, gradients, 60.8.
// Slots never mix Q, K and V, so all that depends on the side is scalar. Other
// heads take the layout of qknorm_rope_paired.hip.

#include "qknorm_rope_device.hpp"

#include <string>
#include <type_traits>

namespace qkn {
namespace {

// The value of the lane H away (H a power of two: lane ^ H).
template <int H>
__device__ __forceinline__ uint32_t from_lane(uint32_t v) {
  const int i = (int)v;
  if constexpr (H == 1) return (uint32_t)__builtin_amdgcn_update_dpp(0, i, 0xB1, 0xF, 0xF, false);   // quad_perm 1,0,3,2
  if constexpr (H == 2) return (uint32_t)__builtin_amdgcn_update_dpp(0, i, 0x4E, 0xF, 0xF, false);   // quad_perm 2,3,0,1
  if constexpr (H == 4) {   // row_shl:4 into banks 0 and 2, row_shr:4 into banks 1 and 3
    const int up = __builtin_amdgcn_update_dpp(0, i, 0x104, 0xF, 0x5, false);
    return (uint32_t)__builtin_amdgcn_update_dpp(up, i, 0x114, 0xF, 0xA, false);
  }
  if constexpr (H == 8) return (uint32_t)__builtin_amdgcn_update_dpp(0, i, 0x128, 0xF, 0xF, false);  // row_ror:8
  if constexpr (H == 16) {
    const auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return threadIdx.x & 16 ? p[0] : p[1];
  }
  const auto p = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return threadIdx.x & 32 ? p[0] : p[1];
}
template <int H, int VW>
__device__ __forceinline__ void fetch(const float (&z)[VW], float (&p)[VW]) {
#pragma unroll
  for (int e = 0; e < VW; ++e) p[e] = __uint_as_float(from_lane<H>(__float_as_uint(z[e])));
}
template <int H, int VW>
__device__ __forceinline__ void fetch(const double (&z)[VW], double (&p)[VW]) {
#pragma unroll
  for (int e = 0; e < VW; ++e) {
    const uint64_t u = __builtin_bit_cast(uint64_t, z[e]);
    p[e] = __builtin_bit_cast(double, (uint64_t)from_lane<H>((uint32_t)(u >> 32)) << 32 | from_lane<H>((uint32_t)u));
  }
}

// A lane's chunk of a head and its part in the rotation.
template <int VW, bool INTER>
struct Chunk1 {
  static constexpr int TW = INTER ? VW / 2 : VW;   // angles of a chunk
  int col;           // first column in the head
  int tab;           // offset of its angles in a table row
  bool turned;       // rotated
  uint32_t flip;     // sign bit for the sine: the first member of a pair subtracts
  __device__ __forceinline__ Chunk1(int lane_in_head, int rot, int half_lanes) {
    col = lane_in_head * VW;
    turned = col < rot;
    tab = !turned ? 0 : INTER ? col / 2 : (lane_in_head & (half_lanes - 1)) * VW;
    flip = !INTER && lane_in_head < half_lanes ? 0x80000000u : 0u;
  }
};

// cos and sin for a lane's chunk at one position (half-split: the sine with
// the sign its member takes). A position outside the table gives NaN, which
// reaches every rotated column of the token.
// AXES: positions on several axes, gathered by the wave and read from LDS.
template <class IO, bool INTER, bool AXES>
struct Turn {
  static constexpr int VW = IO::kVW;
  static constexpr int TW = Chunk1<VW, INTER>::TW;
  static constexpr int kRounds = AXES ? VW / 2 : 1;        // 64 lanes hold a head: at most 64 VW / 2 angles
  static constexpr int kLds = AXES ? 2 * 64 * kRounds : 1;   // floats a wave
  float c[TW], s[TW];
  AxisAngles own;
  bool in;
  // A token's position or positions, to be loaded before its rows: the angles'
  // addresses wait for them.
  struct Where {
    int64_t pos;
    AxisAngles::Positions all;
    template <class Args>
    __device__ __forceinline__ void load(const Args& a, int64_t t) {
      if constexpr (AXES)
        all.load(a, t);
      else
        pos = load_uniform(a.positions + t);
    }
  };
  template <class Args>
  __device__ __forceinline__ void load(const Args& a, const Where& w, const Chunk1<VW, INTER>& at, uint32_t axes) {
    if constexpr (AXES) {
      own.load(a, w.all, axes);
    } else {
      in = w.pos >= 0 && w.pos < a.n_positions;
      const float* row = a.cos_sin + (in ? w.pos : 0) * a.ld_table;
      load_bytes<TW * 4, false>(reinterpret_cast<const char*>(row + at.tab), reinterpret_cast<uint32_t*>(c));
      load_bytes<TW * 4, false>(reinterpret_cast<const char*>(row + (a.rot >> 1) + at.tab), reinterpret_cast<uint32_t*>(s));
    }
  }
  template <class Args>
  __device__ __forceinline__ void settle(const Args& a, int64_t t, const Chunk1<VW, INTER>& at, float* lds) {
    if constexpr (AXES) {
      own.template put<kRounds>(a, t, lds);
#pragma unroll
      for (int e = 0; e < TW; ++e) {
        c[e] = lds[at.tab + e];
        s[e] = lds[kSinAt(kRounds) + at.tab + e];
      }
    } else if (!in) {
      keep_branch();
#pragma unroll
      for (int e = 0; e < TW; ++e) c[e] = s[e] = __builtin_nanf("");
    }
    if constexpr (!INTER) {
#pragma unroll
      for (int e = 0; e < TW; ++e) s[e] = __uint_as_float(__float_as_uint(s[e]) ^ at.flip);
    }
  }
};

// Rotates a lane's chunk (BACK: by the opposite angle, the transposed map that
// gradients take). half_lanes: lanes between the members of a pair. With MAG,
// `mag` gets the magnitudes that each result is the sum of.
template <bool BACK, bool MAG, class F, int VW, class IO, bool INTER, bool AXES>
__device__ __forceinline__ void rotate_chunk(F (&z)[VW], const Turn<IO, INTER, AXES>& t, const Chunk1<VW, INTER>& at,
                                             int half_lanes, bool partial, float (&mag)[VW]) {
  F y[VW], p[VW];
  if constexpr (INTER) {
#pragma unroll
    for (int i = 0; i < VW / 2; ++i) {
      const F c = t.c[i], s = BACK ? -t.s[i] : t.s[i];
      y[2 * i] = z[2 * i] * c - z[2 * i + 1] * s;
      y[2 * i + 1] = z[2 * i + 1] * c + z[2 * i] * s;
      p[2 * i] = z[2 * i + 1];
      p[2 * i + 1] = z[2 * i];
    }
  } else {
    switch (half_lanes) {   // uniform over the launch
      case 8: fetch<8>(z, p); break;
      case 4: fetch<4>(z, p); break;
      case 16: fetch<16>(z, p); break;
      case 2: fetch<2>(z, p); break;
      case 1: fetch<1>(z, p); break;
      default: fetch<32>(z, p); break;
    }
#pragma unroll
    for (int e = 0; e < VW; ++e) y[e] = z[e] * (F)t.c[e] + p[e] * (F)(BACK ? -t.s[e] : t.s[e]);
  }
  if constexpr (MAG) {
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      const int i = INTER ? e / 2 : e;
      const float m = __builtin_fmaf(__builtin_fabsf((float)z[e]), __builtin_fabsf(t.c[i]),
                                     __builtin_fabsf((float)p[e]) * __builtin_fabsf(t.s[i]));
      mag[e] = partial && !at.turned ? mag[e] : m;
    }
  }
#pragma unroll
  for (int e = 0; e < VW; ++e) z[e] = partial && !at.turned ? z[e] : y[e];
}

// The largest over the 32 / VW lanes that hold a block.
template <int VW>
__device__ __forceinline__ uint32_t block_max(uint32_t m) {
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xB1, 0xF, 0xF, false));
  m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4E, 0xF, 0xF, false));
  if (VW == 4) m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x141, 0xF, 0xF, false));
  return m;
}
template <class MX, int VW>
struct Coded {
  Codes<MX, VW> codes;
  int byte;
};

// The largest magnitude of a lane's values, NaN where one of them is.
template <int VW>
__device__ __forceinline__ float largest(const float (&f)[VW]) {
  float m = __builtin_fabsf(f[0]);
#pragma unroll
  for (int e = 1; e < VW; e += 2)
    m = __builtin_elementwise_maximum(__builtin_elementwise_maximum(m, __builtin_fabsf(f[e])),
                                      __builtin_fabsf(f[(e + 1) % VW]));
  return m;
}

// The codes of a lane's values.
template <class MX, int VW>
__device__ __forceinline__ Coded<MX, VW> quantize(const float (&f)[VW]) {
  Coded<MX, VW> q;
  q.byte = scale_byte<MX>(block_max<VW>(__float_as_uint(largest(f)) & 0x7FFFFFFFu));
  const float inv = over_scale(q.byte);
  float a[VW];
#pragma unroll
  for (int e = 0; e < VW; ++e) a[e] = MX::saturated(f[e] * inv);
  if (__builtin_amdgcn_ballot_w64(q.byte == 0xFF) != 0) {
    keep_branch();
#pragma unroll
    for (int e = 0; e < VW; ++e) a[e] = q.byte == 0xFF ? 0.0f : a[e];
  }
  q.codes = codes_of<MX, VW>(a);
  return q;
}

// The codes of values known to within kUnsure of `mag`: true if every value
// within that distance has them (in this lane's share of its block). A value and
// both ends of its interval are of one sign, or their codes differ; 0 is its own
// interval where mag is 0.
constexpr float kUnsure = 0x1.4p-20f;
template <class MX, int VW>
__device__ __forceinline__ bool quantize_sure(const float (&f)[VW], const float (&mag)[VW], Coded<MX, VW>& q) {
  const float top = __uint_as_float(block_max<VW>(__float_as_uint(largest(f)) & 0x7FFFFFFFu));
  const float far = __uint_as_float(block_max<VW>(__float_as_uint(largest(mag)) & 0x7FFFFFFFu));
  const float most = __builtin_fmaf(far, kUnsure, top), least = __builtin_fmaf(far, -kUnsure, top);
  const uint32_t mh = __float_as_uint(most) & 0x7FFFFFFFu;
  q.byte = scale_byte<MX>(mh);
  if (mh >= 0x7F800000u || scale_byte<MX>(least > 0.0f ? __float_as_uint(least) : 0u) != q.byte) return false;
  const float inv = over_scale(q.byte), width = kUnsure * inv;
  float lo[VW], hi[VW];
#pragma unroll
  for (int e = 0; e < VW; ++e) {
    const float v = MX::saturated(f[e] * inv), w = mag[e] * width;
    hi[e] = v + w;
    lo[e] = v - w;
  }
  q.codes = codes_of<MX, VW>(hi);
  return q.codes == codes_of<MX, VW>(lo);
}

// A lane's normalized and rotated chunk formed in float64 and rounded to odd,
// four elements at a time to keep registers for waves.
template <class IO, bool INTER, bool AXES>
__device__ __forceinline__ void exact_chunk(const RopeArgs& a, const char* x, const char* gamma, int64_t pos, bool turns,
                                            const Chunk1<IO::kVW, INTER>& at, const float* lds, int L,
                                            float (&f)[IO::kVW]) {
  constexpr int VW = IO::kVW;
  constexpr int GB = VW * IO::kGBytes;
  float v[VW], g[VW];
  {
    Piece<16> w;
    load_bytes<16, false>(x, w.w);
    widen<IO, VW>(w.w, v);
    if (gamma) {
      Piece<GB> wg;
      load_bytes<GB, false>(gamma, wg.w);
      widen_gamma<IO, VW>(wg.w, g);
    }
  }
  double r = 1.0;
  if (gamma) {
    double ss = 0.0;
#pragma unroll
    for (int e = 0; e < VW; ++e) ss = __builtin_fma((double)v[e], (double)v[e], ss);
    ss = group_sum_d(ss, L);
    // (head_dim is a power of two in this layout.) The hardware's estimate and two Newton
    // steps instead of a division and a square root, which take 60 instructions more. An
    // estimate of 0 stays: m is infinite, where a step would make NaN of 0 m
    const double m = __builtin_fma(ss, (double)a.inv_div, (double)a.eps);
    r = __builtin_amdgcn_rsq(m);
    const double finite = r > 0.0 ? m : 0.0;
#pragma unroll
    for (int k = 0; k < 2; ++k) r = __builtin_fma(r * 0.5, __builtin_fma(-finite * r, r, 1.0), r);
  }
  bool in = false;
  const float* row = nullptr;
  if (!AXES && turns) {
    in = pos >= 0 && pos < a.n_positions;
    row = a.cos_sin + (in ? pos : 0) * a.ld_table + at.tab;
  }
#pragma unroll 1
  for (int e0 = 0; e0 < VW; e0 += 4) {
    double z[4], p[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float one = VW > 4 && e0 ? v[(k + 4) % VW] : v[k];
      z[k] = one;
      if (gamma) z[k] = z[k] * (VW > 4 && e0 ? g[(k + 4) % VW] : g[k]) * r;
    }
    if (turns) {
      if constexpr (INTER) {
#pragma unroll
        for (int k = 0; k < 4; ++k) p[k] = z[k ^ 1];
      } else {
        switch (a.half_lanes) {
          case 8: fetch<8>(z, p); break;
          case 4: fetch<4>(z, p); break;
          case 16: fetch<16>(z, p); break;
          case 2: fetch<2>(z, p); break;
          case 1: fetch<1>(z, p); break;
          default: fetch<32>(z, p); break;
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = INTER ? (e0 + k) >> 1 : e0 + k;
        double c, sn;
        if constexpr (AXES) {
          c = lds[at.tab + i], sn = lds[kSinAt(Turn<IO, INTER, true>::kRounds) + at.tab + i];
        } else {
          c = in ? row[i] : __builtin_nanf(""), sn = in ? row[(a.rot >> 1) + i] : __builtin_nanf("");
        }
        const bool first = INTER ? (k & 1) == 0 : at.flip != 0;   // of its pair: the sine is subtracted
        const double y = z[k] * c + p[k] * (first ? -sn : sn);
        p[k] = at.turned ? y : z[k];
      }
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) p[k] = z[k];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float one = round_to_odd(p[k]);
      if (VW > 4 && e0)
        f[(k + 4) % VW] = one;
      else
        f[k] = one;
    }
  }
}

// The forward pass (MODE ROPE_FORWARD: Q and K rows to y) and the append
// calls (Q to y, K and V into the cache). A wave takes one token's next S
// slots of one side; which, its number says (a.groups waves per token). All of
// a wave's rows are loaded before the first is used, and the angles serve all
// its slots.
// 8192 tokens of 40 + 8 + 8 bf16 heads of 128 into a 4-bit cache: 60.4 us, 4.1
// TB/s, 58.1 without the cached values as rows; Q's launch 33 us runs at 5.1
// TB/s, K's and V's 27 us issues 449 vector instructions a wave in 60% of the
// cycles, beside 81 MB of traffic. Into a cache of bf16 rows 42.0 us, 5.7 TB/s. Into an
// 8-bit cache, on three axes, 67.2: Q's launch 37 us, K's and V's 30 (566 vector
// instructions a wave, 15 us of issue, 63% of the busy cycles; 87 MB, 14 us).
// Apart, because one kernel for both took the registers of the longer one:
// 70 us. The paired layout is faster only for a cache of rows and about a
// thousand tokens (10.7 us against 11.7).
template <class IO, int S, bool INTER, int MODE, bool AXES>
__global__ void __launch_bounds__(64 * kRopeWaves) qknorm_rope_rows(const std::conditional_t<AXES, RopeAxesArgs, RopeArgs> a) {
  constexpr int VW = IO::kVW;
  constexpr bool CODES = MODE == ROPE_APPEND_MXFP4 || MODE == ROPE_APPEND_MXFP8;
  using MX = std::conditional_t<MODE == ROPE_APPEND_MXFP8, Mx8, Mx4>;
  constexpr int GB = VW * IO::kGBytes;
  constexpr uint32_t XR = 16;
  const int lane = threadIdx.x & 63;
  // each run of 8 * XR blocks transposed: the hardware deals blocks to the 8
  // XCDs in turn, and XR consecutive ones (tokens side by side in the cache's
  // pages) then meet in one L2
  uint32_t block = blockIdx.x;
  if (block < (gridDim.x & ~(8u * XR - 1)))
    block = (block & ~(8u * XR - 1)) | ((block & 7) * XR) | ((block >> 3) & (XR - 1));
  const uint32_t unit = block * kRopeWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (unit >= a.units) return;
  const uint32_t t0 = over(unit, a.by_groups);
  const int group = unit - t0 * a.by_groups.d;
  const int c = group < a.first[1] ? 0 : MODE != ROPE_FORWARD && group >= a.first[2] ? 2 : 1;   // Q, K or V
  const RopeSide& o = a.side[c];
  const int L = 1 << a.log2_lanes;
  const int hw = 64 >> a.log2_lanes;
  const int head0 = (group - a.first[c]) * S * hw + (lane >> a.log2_lanes);   // of the first slot
  const Chunk1<VW, INTER> at(lane & (L - 1), a.rot, a.half_lanes);
  const bool partial = a.rot < a.head_dim;
  const bool turns = a.rot != 0 && c != 2;
  using T = Turn<IO, INTER, AXES>;
  __shared__ __align__(16) float angles[kRopeWaves * T::kLds];
  float* const lds = angles + (threadIdx.x >> 6) * T::kLds;
  const uint32_t axes = AXES && turns ? lane_axes(a) : 0;

  const char* gamma = static_cast<const char*>(c == 2 ? nullptr : o.gamma);
  Piece<GB> gam;   // of the first slot: of all where heads share it
  if (gamma) load_bytes<GB, false>(gamma + ((head0 < o.heads ? head0 : 0) * a.gstride + at.col) * IO::kGBytes, gam.w);
  uint32_t off[S];
#pragma unroll
  for (int i = 0; i < S; ++i) {
    const int head = head0 + i * hw;
    off[i] = (uint32_t)((head < o.heads ? head : 0) * a.head_dim + at.col) * IO::kBytes;   // idle lanes: the first head
  }

  // Slot i's results (codes in q, for a cache of them) to where they go.
  const auto store = [&](int i, bool on, float (&f)[VW], const Coded<MX, VW>& q, int64_t t, int64_t place) {
    const int64_t head = head0 + i * hw;
    if (MODE != ROPE_FORWARD && c != 0) {
      const int64_t page = place >> a.log2_page, in = place & (((int64_t)1 << a.log2_page) - 1);
      char* p = a.cache[c - 1] + page * a.page_stride + in * a.token_stride + head * a.head_stride;
      if constexpr (CODES) {
        char* sc = a.scales[c - 1] + page * a.scale_page_stride + in * (a.head_dim >> 5) + head * a.scale_head_stride;
        if (on) {
          store_bytes<VW * MX::kBits / 8>(p + at.col * MX::kBits / 8, q.codes.w);
          if ((lane & (32 / VW - 1)) == 0) sc[at.col >> 5] = (char)q.byte;
        }
        if (o.y) code_values<MX, VW>(q.codes, q.byte, f);
      } else {
        Piece<16> w;
        narrow<IO, VW>(f, w.w);
        if (on) store_bytes<16>(p + at.col * IO::kBytes, w.w);
      }
    }
    if (o.y) {
      Piece<16> w;
      narrow<IO, VW>(f, w.w);
      if (on) store_bytes<16>(static_cast<char*>(o.y) + t * o.ldy * IO::kBytes + (head * a.head_dim + at.col) * IO::kBytes, w.w);
    }
  };

  for (int64_t t = t0; t < a.T; t += a.tokens) {
    uint32_t unsure = 0;   // slots whose codes float32 leaves open
    // A row that holds no token is worked like the others, and not stored: its
    // slot, waited for first, would hold up all that follows.
    int64_t place = 0;
    if constexpr (MODE != ROPE_FORWARD) place = load_uniform(a.slots + t);
    typename T::Where where;
    if (turns) where.load(a, t);
    Piece<16> x[S];
#pragma unroll
    for (int i = 0; i < S; ++i)
      load_bytes<16, true>(static_cast<const char*>(o.x) + t * o.ldx * IO::kBytes + off[i], x[i].w);
    T turn;
    if (turns) {
      turn.load(a, where, at, axes);
      turn.settle(a, t, at, lds);
    }
    const bool live = MODE == ROPE_FORWARD || (place >= 0 && place < a.n_tokens_held);

#pragma unroll
    for (int i = 0; i < S; ++i) {
      const bool on = head0 + i * hw < o.heads;
      if (i > 0 && __builtin_amdgcn_ballot_w64(on) == 0) break;   // the side's last slot is done
      if (i > 0 && gamma && a.gstride)
        load_bytes<GB, false>(gamma + ((on ? head0 + i * hw : 0) * a.gstride + at.col) * IO::kGBytes, gam.w);
      float f[VW];
      widen<IO, VW>(x[i].w, f);
      float mag[VW];
      bool ranged = true;   // float32 held the head's sum and its products (see below)
      if (gamma) {
        float ss = 0.0f;
#pragma unroll
        for (int e = 0; e < VW; ++e) ss = __builtin_fmaf(f[e], f[e], ss);
        ss = group_sum(ss, L);
        const float r = rms_factor(ss, a.inv_div, a.eps);
        ranged = r > 0.0f && r <= MX::kMostFactor;
        float g[VW];
        widen_gamma<IO, VW>(gam.w, g);
#pragma unroll
        for (int e = 0; e < VW; ++e) f[e] = (f[e] * g[e]) * r;
      }
      if (CODES) {
#pragma unroll
        for (int e = 0; e < VW; ++e) mag[e] = __builtin_fabsf(f[e]);
      }
      if (turns) rotate_chunk<false, CODES>(f, turn, at, a.half_lanes, partial, mag);

      Coded<MX, VW> q;
      if (CODES && c != 0) {
        if (c == 2) {
          q = quantize<MX, VW>(f);
        } else {
          const bool sure = quantize_sure<MX, VW>(f, mag, q);
          if (__builtin_amdgcn_ballot_w64(!(sure && ranged)) != 0) {
            unsure |= 1u << i;
            continue;
          }
        }
      }
      store(i, on && live, f, q, t, place);
    }

    if constexpr (CODES) {
      // A key's float32 value is within 16 u of the magnitudes it is the sum of (r
      // within 11 u: a chain of 8 squares, 6 butterfly adds, the factor; then 4
      // roundings), u = 2^-24. kUnsure is 20 u: one more for the rounding of the
      // interval's ends, and 3 u of the lowest border there is, 2^-102 (8 bits:
      // 2^-110), are more than what subnormal roundings of 2^-150 come to where r is
      // at most 2^24 (2^16): 2^-126 for each of the two that make a value. (Twice as
      // wide, 8 bits take 1 us longer.) It is so where the sum is finite (r > 0).
      // Where a border of the codes or of the scale lies that near to one (in 0.4% of
      // the slots, with 8 bits in 6%), or r is out of that range, the slot is formed
      // again in float64, so that every code is the one exact arithmetic gives and
      // does not hang on the order of a sum.
      // Here, behind the others, where little else is held in registers (in
      // float64 throughout, 8192 tokens took 69 us).
#pragma unroll 1
      for (int i = 0; live && unsure != 0; ++i, unsure >>= 1) {
        if (!(unsure & 1)) continue;
        const int head = head0 + i * hw;
        const bool on = head < o.heads;
        float f[VW];
        exact_chunk<IO, INTER, AXES>(
            a, static_cast<const char*>(o.x) + t * o.ldx * IO::kBytes + (int64_t)((on ? head : 0) * a.head_dim + at.col) * IO::kBytes,
            gamma ? gamma + ((on ? head : 0) * a.gstride + at.col) * IO::kGBytes : nullptr,
            where.pos, turns, at, lds, L, f);
        const Coded<MX, VW> q = quantize<MX, VW>(f);
        store(i, on, f, q, t, place);
      }
    }
  }
}

// Gradients. With g the incoming gradient turned back by the rotation, xr =
// x * r and gg = g * gamma: dgamma_j = sum over tokens (and heads sharing
// gamma) of g_j xr_j, and dx = r (gg - xr mean(gg xr)). x and dy are read
// once, dx written once; everything between stays in registers. A wave keeps
// one slot of heads for all its tokens, so its share of dgamma stays in
// registers too and leaves as one partial row per block (its waves added in
// LDS in a fixed order); qknorm_rope_grad_sum adds the rows in a fixed order,
// so the gradients do not change from run to run. The next token's loads are
// issued before the current one is worked on. 8192 tokens x 48 heads x 128
// bf16 columns: 59.5 us with the sums (56 and 5 traced one by one), 5.1 TB/s
// where a copy of one stream reaches 6.06; 32 float32 heads 72.9 us, 5.6 TB/s.
template <class IO, bool INTER, bool AXES>
__global__ void __launch_bounds__(64 * kGradWaves) qknorm_rope_grad(const std::conditional_t<AXES, RopeGradAxesArgs, RopeGradArgs> a) {
  constexpr int VW = IO::kVW;
  constexpr int GB = VW * IO::kGBytes;
  __shared__ float red[kGradWaves * 64 * VW];
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
  const Chunk1<VW, INTER> at(lane & (L - 1), a.rot, a.half_lanes);
  const bool partial = a.rot < a.head_dim;
  using T = Turn<IO, INTER, AXES>;
  __shared__ __align__(16) float angles[kGradWaves * T::kLds];
  float* const lds = angles + wave * T::kLds;
  const uint32_t axes = lane_axes(a);
  const uint32_t off = (uint32_t)(hc * a.head_dim + at.col) * IO::kBytes;

  float g[VW], sum[VW];
  {
    Piece<GB> p;
    load_bytes<GB, false>(static_cast<const char*>(o.gamma) + (hc * a.gstride + at.col) * IO::kGBytes, p.w);
    widen_gamma<IO, VW>(p.w, g);
#pragma unroll
    for (int e = 0; e < VW; ++e) sum[e] = 0.0f;
  }

  struct In {
    Piece<16> x, dy;
    T turn;
  };
  const auto load = [&](In& in, int64_t t) {
    load_bytes<16, true>(static_cast<const char*>(o.x) + t * o.ldx * IO::kBytes + off, in.x.w);
    load_bytes<16, true>(static_cast<const char*>(o.dy) + t * o.lddy * IO::kBytes + off, in.dy.w);
    if (a.rot) {
      typename T::Where where;
      where.load(a, t);
      in.turn.load(a, where, at, axes);
    }
  };
  const auto work = [&](In& in, int64_t t) {
    float x[VW], y[VW], gg[VW];
    widen<IO, VW>(in.x.w, x);
    widen<IO, VW>(in.dy.w, y);
    if (a.rot) {
      in.turn.settle(a, t, at, lds);
      rotate_chunk<true, false>(y, in.turn, at, a.half_lanes, partial, gg);
    }
    float ss = 0.0f, dot = 0.0f;
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      ss = __builtin_fmaf(x[e], x[e], ss);
      gg[e] = y[e] * g[e];
      dot = __builtin_fmaf(gg[e], x[e], dot);
    }
    group_sum_qk(ss, dot, L);
    const float r = rms_factor(ss, a.inv_div, a.eps);
    const float mean = (dot * r) * a.inv_div;
    float d[VW];
#pragma unroll
    for (int e = 0; e < VW; ++e) {
      const float xr = x[e] * r;
      sum[e] = __builtin_fmaf(y[e], xr, sum[e]);
      d[e] = r * __builtin_fmaf(-xr, mean, gg[e]);
    }
    Piece<16> p;
    narrow<IO, VW>(d, p.w);
    if (on) store_bytes<16>(static_cast<char*>(o.dx) + t * o.lddx * IO::kBytes + off, p.w);
  };
  each_token<In>((int64_t)blockIdx.x * kGradWaves + wave, (int64_t)a.workers * kGradWaves, a.T, load, work);

  if (!o.dgamma) return;
#pragma unroll
  for (int e = 0; e < VW; ++e) red[(wave * VW + e) * 64 + lane] = sum[e];
  __syncthreads();
  // Shared gamma: one row per (slot, worker), the slot's heads added too;
  // otherwise one row per (head, worker).
  const bool shared = a.gstride == 0;
  const int live = min(hw, o.heads - (s - a.first[c]) * hw);   // heads of this slot
  for (int i = threadIdx.x; i < VW * 64; i += 64 * kGradWaves) {
    const int l = i & 63, e = i >> 6;
    const int lh = l >> a.log2_lanes;
    if (shared ? lh != 0 : lh >= live) continue;
    float all = 0.0f;
    for (int h = 0; h < (shared ? live : 1); ++h)
      for (int w = 0; w < kGradWaves; ++w) all += red[(w * VW + e) * 64 + l + (h << a.log2_lanes)];
    const int global_head = (c ? a.side[0].heads : 0) + (s - a.first[c]) * hw + lh;
    const int64_t row = shared ? (int64_t)s * a.workers + blockIdx.x : (int64_t)global_head * a.workers + blockIdx.x;
    a.partial[row * a.head_dim + (l & (L - 1)) * VW + e] = all;
  }
}

// dgamma from the partial rows: 32 columns and 32 row groups per block, sums
// in float64 (a few thousand terms), groups joined in LDS.
__global__ void __launch_bounds__(1024) qknorm_rope_grad_sum(const RopeGradArgs a) {
  __shared__ double red[32][33];
  const bool shared = a.gstride == 0;
  const int o = blockIdx.y;
  const int c = shared ? o : (o >= a.side[0].heads ? 1 : 0);
  float* dst = a.side[c].dgamma;
  if (!dst) return;
  const int col = blockIdx.x * 32 + (threadIdx.x & 31);
  const int group = threadIdx.x >> 5;
  int64_t row0, n;
  if (shared) {
    row0 = (int64_t)a.first[c] * a.workers;
    n = (int64_t)((c ? a.n_slots : a.first[1]) - a.first[c]) * a.workers;
  } else {
    row0 = (int64_t)o * a.workers;
    n = a.workers;
    dst += (int64_t)(o - (c ? a.side[0].heads : 0)) * a.gstride;
  }
  double sum = 0.0;
  if (col < a.head_dim) {
    const float* p = a.partial + row0 * a.head_dim + col;
#pragma unroll 4
    for (int64_t i = group; i < n; i += 32) sum += (double)p[i * a.head_dim];
  }
  red[group][threadIdx.x & 31] = sum;
  __syncthreads();
  if (threadIdx.x < 32 && col < a.head_dim) {
    double all = 0.0;
    for (int g = 0; g < 32; ++g) all += red[g][threadIdx.x];
    dst[col] = (float)all;
  }
}

template <class IO, bool INTER, int MODE, bool AXES>
const void* pick_slots(int slots) {
  switch (slots) {
    case 1: return reinterpret_cast<const void*>(qknorm_rope_rows<IO, 1, INTER, MODE, AXES>);
    case 2: return reinterpret_cast<const void*>(qknorm_rope_rows<IO, 2, INTER, MODE, AXES>);
    case 3: return reinterpret_cast<const void*>(qknorm_rope_rows<IO, 3, INTER, MODE, AXES>);
    case 4: return reinterpret_cast<const void*>(qknorm_rope_rows<IO, 4, INTER, MODE, AXES>);
  }
  return nullptr;
}

template <class IO, bool INTER, bool AXES>
const void* pick_mode(int mode, int slots) {
  if (mode == ROPE_FORWARD) return pick_slots<IO, INTER, ROPE_FORWARD, AXES>(slots);
  if constexpr (IO::kBytes > 1) {
    if (mode == ROPE_APPEND_ROWS) return pick_slots<IO, INTER, ROPE_APPEND_ROWS, AXES>(slots);
    if (mode == ROPE_APPEND_MXFP8) return pick_slots<IO, INTER, ROPE_APPEND_MXFP8, AXES>(slots);
    return pick_slots<IO, INTER, ROPE_APPEND_MXFP4, AXES>(slots);
  }
  return nullptr;
}

template <class IO>
const void* pick_turn(int mode, bool inter, bool axes, int slots) {
  if (axes) return inter ? pick_mode<IO, true, true>(mode, slots) : pick_mode<IO, false, true>(mode, slots);
  return inter ? pick_mode<IO, true, false>(mode, slots) : pick_mode<IO, false, false>(mode, slots);
}

const void* rope_kernel(int mode, int dtype, bool inter, bool axes, const RopePlan& p) {
  if (!p.whole) return rope_paired_kernel(mode, dtype, inter, axes, p);
  switch (dtype) {
    case kDtypeBF16: return pick_turn<BF16>(mode, inter, axes, p.slots);
    case kDtypeF32: return pick_turn<F32>(mode, inter, axes, p.slots);
    default: return pick_turn<FP8>(mode, inter, axes, p.slots);
  }
}

template <class IO>
const void* pick_grad_turn(bool inter, bool axes) {
  if (axes)
    return inter ? reinterpret_cast<const void*>(qknorm_rope_grad<IO, true, true>)
                 : reinterpret_cast<const void*>(qknorm_rope_grad<IO, false, true>);
  return inter ? reinterpret_cast<const void*>(qknorm_rope_grad<IO, true, false>)
               : reinterpret_cast<const void*>(qknorm_rope_grad<IO, false, false>);
}

const void* rope_grad_kernel(int dtype, bool inter, bool axes, const RopePlan& p) {
  if (!p.whole) return rope_paired_grad_kernel(dtype, inter, axes, p);
  return dtype == kDtypeBF16 ? pick_grad_turn<BF16>(inter, axes) : pick_grad_turn<F32>(inter, axes);
}

int launched(hipError_t e, std::string* err) {
  if (e == hipSuccess) return 0;
  *err = std::string("kernel launch: ") + hipGetErrorString(e);
  return (int)e;
}

}  // namespace

constexpr int64_t kRopeMostBlocks = (int64_t)1 << 22;

static int launch_rows(int mode, int dtype, bool inter, const RopePlan& p, RopeAxesArgs a, void* stream, std::string* err) {
  const void* fn = rope_kernel(mode, dtype, inter, a.axes.n > 0, p);
  if (!fn) {
    *err = "no kernel compiled for this plan";
    return (int)hipErrorInvalidValue;
  }
  int64_t blocks = (a.T + p.tokens - 1) / p.tokens;
  unsigned gy = 1, threads = (unsigned)(64 * p.waves * p.tokens);
  if (p.whole) {
    // units: waves of the first a.tokens tokens; the rest of the tokens loop
    // (a launch holds fewer than 2^32 threads)
    const int64_t most = (grid_cap() < kRopeMostBlocks ? grid_cap() : kRopeMostBlocks) * kRopeWaves / p.groups;
    a.tokens = (int)(a.T < most ? a.T : most > 0 ? most : 1);
    a.units = (uint32_t)((int64_t)a.tokens * p.groups);
    a.by_groups = divisor((uint32_t)p.groups);
    blocks = ((int64_t)a.units + kRopeWaves - 1) / kRopeWaves;
    threads = 64 * kRopeWaves;
  } else {
    // gy blocks take a token's slots: the cap holds for their product, down to one token's blocks
    gy = (unsigned)((a.n_slots + p.slots * p.waves - 1) / (p.slots * p.waves));
    const int64_t most = (grid_cap() < kRopeMostBlocks ? grid_cap() : kRopeMostBlocks) / gy;
    // Of bf16 rows a compute unit holds eight waves of three slots. Where there are more,
    // these take several tokens each, in equal numbers, and load the next one's rows before
    // this one's work: 8192 tokens of 32 + 8 heads of 80 on three axes 29.5 us, a wave a
    // token 37.3; heads of 96 34.2 and 39.5, and appended to MXFP8 with one position 51.9
    // and 62.3. Not codes with several axes, whose registers do not suffice for two tokens
    // (74 us, 63.3), nor rows with several axes (41 either way); calls with one position and
    // no MXFP8 keep a wave a token.
    const bool shared = (mode == ROPE_FORWARD && a.axes.n > 0) || (mode == ROPE_APPEND_MXFP8 && a.axes.n == 0);
    const int64_t held = 256 * 8 / ((int64_t)p.waves * p.tokens * gy);
    if (shared && dtype == kDtypeBF16 && p.slots == 3 && held > 0 && blocks > held) {
      const int64_t rounds = (blocks + held - 1) / held;
      blocks = (blocks + rounds - 1) / rounds;
    }
    if (blocks > most) blocks = most > 0 ? most : 1;
  }
  void* kargs[] = {&a};
  return launched(hipLaunchKernel(fn, dim3((unsigned)blocks, gy), dim3(threads), kargs, 0,
                                  static_cast<hipStream_t>(stream)),
                  err);
}

int launch_rope(int mode, int dtype, bool inter, const RopePlan& p, const RopeAxesArgs& args, void* stream,
                std::string* err) {
  if (!p.apart) return launch_rows(mode, dtype, inter, p, args, stream, err);
  // Q by itself, in the row-type kernel (it writes rows only), then K and V
  RopePlan part = p;
  RopeAxesArgs a = args;
  a.side[1].heads = a.side[2].heads = 0;
  a.first[2] = a.first[1];
  part.groups = a.first[1];
  if (const int rc = launch_rows(ROPE_APPEND_ROWS, dtype, inter, part, a, stream, err)) return rc;
  a = args;
  a.side[0].heads = 0;
  a.first[1] = 0;
  a.first[2] = args.first[2] - args.first[1];
  part.groups = p.groups - args.first[1];
  return launch_rows(mode, dtype, inter, part, a, stream, err);
}

int64_t rope_grad_rows(const RopeGradArgs& a) {
  return (int64_t)(a.gstride == 0 ? a.n_slots : a.side[0].heads + a.side[1].heads) * a.workers;
}

int launch_rope_grad(int dtype, bool inter, const RopePlan& p, const RopeGradAxesArgs& args, void* stream,
                     std::string* err) {
  const void* fn = rope_grad_kernel(dtype, inter, args.axes.n > 0, p);
  RopeGradAxesArgs a = args;
  void* kargs[] = {&a};
  const int rc = launched(hipLaunchKernel(fn,
                                          dim3((unsigned)a.workers, (unsigned)a.n_slots), dim3(64 * kGradWaves), kargs,
                                          0, static_cast<hipStream_t>(stream)),
                          err);
  if (rc || !(a.side[0].dgamma || a.side[1].dgamma)) return rc;
  const unsigned outs = a.gstride == 0 ? 2u : (unsigned)(a.side[0].heads + a.side[1].heads);
  return launched(hipLaunchKernel(reinterpret_cast<const void*>(qknorm_rope_grad_sum),
                                  dim3((unsigned)((a.head_dim + 31) / 32), outs), dim3(1024), kargs, 0,
                                  static_cast<hipStream_t>(stream)),
                  err);
}

}  // namespace qkn

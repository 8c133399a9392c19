// Attention over a paged key / value cache held in 4 bits (MXFP4), on gfx950
// (CDNA4).
//
// For query row r of a sequence and the cached tokens t it sees,
// out_r = sum_t softmax_t(scale q_r . k_t) v_t, in one pass over the cache:
// a running maximum m and sum l per row, and an accumulator that is rescaled
// when m grows.
//
// K and V are E2M1 codes with one E8M0 scale per 32 channels. gfx950 widens a
// byte of codes to two bf16 values with its scale applied in one instruction
// (v_cvt_scalef32_pk_bf16_fp4), exactly: a code times a power of two fits
// bf16. So the products run on bf16 MFMA tiles with nothing lost on the K
// and V side; queries are bf16 already; probabilities are rounded to bf16
// (at most half a step, 2^-8 relative, averaged over the tokens), about as much
// as the rounding of the output itself: against float64, outputs are off by
// 0.0023 in the root mean square, 0.0017 with that rounding alone. Scores, m,
// l and the accumulator are float32.
//
// Work layout. A block takes one key head of one sequence, RT tiles of 16
// query rows (rows are query-major: all heads of a group side by side, so a
// decoded token's group shares one read of the cache) and one chunk of the
// cache; its four waves take the chunk's 32-token tiles in turn, each with
// its own m, l and accumulator, joined in LDS at the end. Chunks of one
// sequence are joined by qknorm_attend_join. The scores are formed
// transposed (tokens x rows), so that a lane holds one row's scores: the
// lane's eight tokens are then just the eight k-positions it must hold of the
// second product's operand, and probabilities go from one product to the
// other in registers. Within a tile the order of channels (first product) and
// tokens (second) is free as long as both operands agree; it is chosen so
// that a lane's codes are 16 (K) and 4 (V) consecutive bytes at 128 channels.
//
// What bounds it. Decoding with many blocks: the cache's bytes (64 sequences of
// up to 8192 tokens, 8 key heads of 128 columns: 88.8 us, 83 of them in this
// launch at 4.95 TB/s, where a copy reaches 6.06). One long sequence: each
// wave's chain of a few tiles and the second launch (65536 tokens 21.9 us, 17 +
// 5; 3.3 TB/s). Prompts: 1024 rows a sequence on 8192 tokens, four of them, take
// 644 us, 740 TFLOP/s. The matrix unit is busy for 203 us of it and the vector
// unit (widening, exponentials, masks) for 275, and two waves per SIMD are all
// that the accumulators leave room for; at least 166 us are neither: the blocks
// are 4.3 rounds of what the chip holds (the last round costs 15% by their
// lengths alone), the rest waits. Two of 1024 rows on 4096 tokens: 32 heads of 64
// columns 100 us (466 TFLOP/s), 16 of 256 161 (578).

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <string>

#include "qknorm_device.hpp"
#include "qknorm_internal.hpp"
#include "qknorm_ops.hpp"

namespace qkn {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2_t __attribute__((ext_vector_type(2)));

constexpr int kWaves = 4;
constexpr uint32_t kTopScale = 252;       // largest scale byte of a finite block; above it, NaN
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

template <int SEL>
__device__ __forceinline__ uint32_t widen_pair(uint32_t codes, float scale) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, SEL));
}
__device__ __forceinline__ uint32_t widen_byte(uint32_t codes, float scale, int sel) {
  switch (sel) {   // sel is a constant after unrolling
    case 0: return widen_pair<0>(codes, scale);
    case 1: return widen_pair<1>(codes, scale);
    case 2: return widen_pair<2>(codes, scale);
    default: return widen_pair<3>(codes, scale);
  }
}

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

// Codes and scales of one 32-token tile, as one lane holds them: lane = 16 g
// + m. K: token m of each half, a quarter of its channels (chosen by g). V:
// tokens 4g .. 4g+3 of each half, channels m * D/16 and on.
template <int D>
struct KTile {
  static constexpr int W = D / 32;               // words of codes per half
  static constexpr int S = D == 256 ? 2 : 1;     // scales per half
  uint32_t c[2][W];
  uint32_t s[2][S];
};
template <int D>
struct VTile {
  static constexpr int W = D == 256 ? 2 : 1;     // words of codes per token
  uint32_t c[2][4][W];
  uint32_t s[2][4];                              // the words that hold the scale bytes
};

// Page ids of a tile's two halves (looked up a tile ahead of its loads, which
// wait for them).
struct Pages {
  int id[2];
};
__device__ __forceinline__ Pages find_pages(const AttendArgs& a, const int32_t* table, int tok, int last16) {
  Pages p;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    // past the end of the chunk: its last 16 tokens again, masked later
    const int t = min(tok + 16 * h, last16);
    p.id[h] = load_uniform(table + (t >> a.log2_page));
  }
  return p;
}

// Where a tile's halves lie: byte offsets of their first tokens' codes and
// scales within a key head, in scalar registers (the compiler forms 64-bit
// products on the vector unit even of uniform values, and every address that
// follows would then be a vector pair of its own).
struct Place {
  uint64_t codes[2], scales[2];
  bool lost[2];      // the page does not exist
};
template <int D>
__device__ __forceinline__ Place place_of(const AttendArgs& a, const Pages& pages, int tok, int last16) {
  Place p;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int off = min(tok + 16 * h, last16) & ((1 << a.log2_page) - 1);
    p.lost[h] = (uint32_t)pages.id[h] >= a.n_pages;
    const uint32_t page = p.lost[h] ? 0 : pages.id[h];
    p.codes[h] = uniform64(page * (uint64_t)a.page_stride + (uint32_t)off * (uint64_t)(D / 2));
    p.scales[h] = uniform64(page * (uint64_t)a.scale_page_stride + (uint32_t)off * (uint64_t)(D / 32));
  }
  return p;
}

// A lane's byte offsets into a tile half.
struct LaneOffsets {
  uint32_t kc, ks, vc, vs;
};
template <int D>
__device__ __forceinline__ LaneOffsets lane_offsets(int lane) {
  const uint32_t m = lane & 15, g = lane >> 4;
  LaneOffsets o;
  o.kc = m * (D / 2) + g * (D == 64 ? 8 : 16);
  o.ks = m * (D / 32) + (D == 64 ? g >> 1 : g);
  o.vc = 4 * g * (D / 2) + m * (D / 32);
  o.vs = 4 * g * (D / 32) + (D == 256 ? (m >> 3) * 4 : 0);
  return o;
}

// A global load at a scalar base, a lane's byte offset and a constant. Both
// are hidden from the compiler where they are used: it would otherwise add
// the lane's offset to the loop-invariant part of the base, or widen it to 64
// bits, once for the whole loop, and hold a vector pair for each load.
template <class T>
__device__ __forceinline__ T load_at(uint64_t base, uint32_t offset, int constant) {
  typedef const T __attribute__((address_space(1)))* gptr;
  return *reinterpret_cast<gptr>((base + (uint64_t)offset) + constant);
}
__device__ __forceinline__ uint64_t pinned(uint64_t v) {
  asm volatile("" : "+s"(v));
  return v;
}

template <int D>
__device__ __forceinline__ void load_k(KTile<D>& T, uint64_t codes, uint64_t scales, const Place& at, LaneOffsets& o) {
  asm volatile("" : "+v"(o.kc), "+v"(o.ks));
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint64_t c = pinned(codes + at.codes[h]), s = pinned(scales + at.scales[h]);
    if constexpr (D == 64) {
      const u32x2_t w = load_at<u32x2_t>(c, o.kc, 0);
      T.c[h][0] = w.x, T.c[h][1] = w.y;
      T.s[h][0] = load_at<uint8_t>(s, o.ks, 0);
    } else {
#pragma unroll
      for (int sp = 0; sp < D / 128; ++sp) {
        const u32x4_t w = load_at<u32x4_t>(c, o.kc, 64 * sp);
        T.c[h][4 * sp] = w.x, T.c[h][4 * sp + 1] = w.y, T.c[h][4 * sp + 2] = w.z, T.c[h][4 * sp + 3] = w.w;
        T.s[h][sp] = load_at<uint8_t>(s, o.ks, 4 * sp);
      }
    }
  }
}

template <int D>
__device__ __forceinline__ void load_v(VTile<D>& T, uint64_t codes, uint64_t scales, const Place& at, LaneOffsets& o) {
  asm volatile("" : "+v"(o.vc), "+v"(o.vs));
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint64_t c = pinned(codes + at.codes[h]), s = pinned(scales + at.scales[h]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (D == 64) {
        T.c[h][j][0] = load_at<uint16_t>(c, o.vc, j * (D / 2));
      } else if constexpr (D == 128) {
        T.c[h][j][0] = load_at<uint32_t>(c, o.vc, j * (D / 2));
      } else {
        const u32x2_t w = load_at<u32x2_t>(c, o.vc, j * (D / 2));
        T.c[h][j][0] = w.x, T.c[h][j][1] = w.y;
      }
    }
    // the scale words of the lane's four tokens; the byte is taken in use
    if constexpr (D == 64) {
      const u32x2_t w = load_at<u32x2_t>(s, o.vs, 0);
      T.s[h][0] = w.x, T.s[h][1] = w.x >> 16, T.s[h][2] = w.y, T.s[h][3] = w.y >> 16;
    } else if constexpr (D == 128) {
      const u32x4_t w = load_at<u32x4_t>(s, o.vs, 0);
      T.s[h][0] = w.x, T.s[h][1] = w.y, T.s[h][2] = w.z, T.s[h][3] = w.w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) T.s[h][j] = load_at<uint32_t>(s, o.vs, j * 8);
    }
  }
}

// The channel at which chunk c (8 channels) of lane group g begins.
template <int D>
__device__ __forceinline__ int k_channel(int g, int c) {
  return D == 64 ? 16 * g + 8 * c : 128 * (c >> 2) + 32 * g + 8 * (c & 3);
}

template <int D, int RT>
__global__ void __launch_bounds__(64 * kWaves, RT * D <= 128 ? 3 : 2) qknorm_attend(const AttendArgs a) {
  constexpr int CB = D / 16;                 // 16-channel blocks of the output
  constexpr int LD = D + 4;                  // padded row of the join buffer
  constexpr int KC = D / 32;                 // 8-channel chunks a lane holds of a row
  constexpr bool QL = RT * D >= 256;         // queries in LDS, in fragment order, instead of registers
  constexpr int NP = D == 256 ? 2 : 1;       // 32-channel blocks a lane's outputs lie in
  constexpr bool LATE = RT * D >= 512;       // V is loaded within its tile, after the first product: registers are short
  constexpr int kStep = 32 * kWaves;
  // the join buffer; before the join, where QL, the queries
  __shared__ __align__(16) float red[kWaves * 16 * LD];
  __shared__ float red_m[kWaves * 16], red_l[kWaves * 16];
  static_assert(!QL || RT * KC * 64 * sizeof(Frag) <= sizeof(red), "the queries fit the join buffer");
  Frag* q_lds = reinterpret_cast<Frag*>(red);

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = lane & 15, g = lane >> 4;
  // blocks of one (sequence, key head) lie a multiple of their count apart:
  // on one XCD, whose L2 then holds that head's cache, where it divides by 8
  const uint32_t rest = over(blockIdx.x, a.by_pairs);
  const uint32_t pair = blockIdx.x - rest * a.by_pairs.d;
  const uint32_t tile_rev = over(rest, a.by_splits);
  const int split = rest - tile_rev * a.by_splits.d;
  const int grid_tile = a.row_tiles - 1 - (int)tile_rev;   // long rows first
  const int b = over(pair, a.by_heads);
  const int hk = pair - b * a.heads_k;

  const Sequence seq = sequence(a, b);
  const int32_t* table = a.table + b * a.ld_table;
  // of this key head
  const uint64_t kc = uniform64((uint64_t)a.cache[0] + hk * a.head_stride);
  const uint64_t vc = uniform64((uint64_t)a.cache[1] + hk * a.head_stride);
  const uint64_t ks = uniform64((uint64_t)a.scales[0] + hk * a.scale_head_stride);
  const uint64_t vs = uniform64((uint64_t)a.scales[1] + hk * a.scale_head_stride);
  const int rows = seq.nq * a.group;
  const int heads_q = a.heads_k * a.group;

  for (int r0 = grid_tile * (16 * RT); r0 < rows; r0 += a.row_tiles * (16 * RT)) {
    const int i_first = over(r0, a.by_group);
    const int i_last = over(min(rows, r0 + 16 * RT) - 1, a.by_group);
    const Span sp = span(a, seq, i_first, i_last);
    const int lo_all = see_lo(a, seq, i_last), hi_all = see_hi(a, seq, i_first);   // every row sees these
    const bool joined = sp.chunks > 1 && a.splits > 1;   // partial results: qknorm_attend_join finishes
    if (split > 0 && split >= sp.chunks) continue;       // nothing of the cache left for this block

    // This lane's row of each tile is m. What it sees is needed at the edges
    // alone and formed there.
    const auto limits = [&](int rt, int* lo, int* hi) {
      const int r = r0 + rt * 16 + m;
      const int i = r < rows ? (int)over(r, a.by_group) : 0;
      *lo = see_lo(a, seq, i);
      *hi = r < rows ? see_hi(a, seq, i) : 0;
    };
    Frag q[QL ? 1 : RT][KC];
    if constexpr (QL) __syncthreads();   // the last rows' readers are done
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int r = r0 + rt * 16 + m;
      const bool on = r < rows;
      const int i = on ? (int)over(r, a.by_group) : 0;
      const int head = hk * a.group + (on ? r - i * a.group : 0);
      const char* p = static_cast<const char*>(a.q) + ((int64_t)(seq.q0 + i) * a.ldq + (int64_t)head * D) * 2;
      if (QL && rt % kWaves != wave) continue;
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        u32x4_t w = {0, 0, 0, 0};
        if (on) w = *reinterpret_cast<const u32x4_t*>(p + k_channel<D>(g, c) * 2);
        const Frag f = {{w.x, w.y, w.z, w.w}};
        if constexpr (QL) {
          q_lds[(rt * KC + c) * 64 + lane] = f;
        } else {
          q[rt][c] = f;
        }
      }
    }
    if constexpr (QL) __syncthreads();
    // acc_l: the sums of the probabilities, by products with a row of ones
    float run_m[RT];
    f32x4_t acc[RT][CB], acc_l[RT];
    uint32_t poison = 0;                  // (tile, block of channels) that NaN values reached
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      run_m[rt] = kNothing;
      acc_l[rt] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int cb = 0; cb < CB; ++cb) acc[rt][cb] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    }

    LaneOffsets offs = lane_offsets<D>(lane);
    int q_at = lane;   // where this lane's query fragments lie in LDS
    int last16 = 0;    // the chunk's last 16 tokens

    // One 32-token tile. Each part of the wave's next one is loaded as soon as
    // the registers of this one's are free: K after the first product, V after
    // the second (LATE: this tile's V, after the first). Loads past the end of
    // the chunk read its last tokens again (the next chunk's would be read from
    // memory for nothing: one tile in seven of a 768-token chunk).
    const auto tile = [&](KTile<D>& K, VTile<D>& V, Place& at, Pages& ahead, int tok, int end) {
      // scores, transposed: lane (m, g) gets tokens 16h + 4g + i of row m
      f32x4_t s[RT][2];
      uint32_t top_ks = 0;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int x = 0; x < KTile<D>::S; ++x) top_ks = max(top_ks, K.s[h][x]);
      const bool any_kbad = __builtin_amdgcn_ballot_w64(top_ks > kTopScale) != 0 || at.lost[0] || at.lost[1];
      // KH halves at a time: with queries in LDS both, so that a fragment is read once for them
      constexpr int KH = QL && RT * D <= 512 && D <= 128 ? 2 : 1;
#pragma unroll
      for (int h0 = 0; h0 < 2; h0 += KH) {
        Frag kf[KH][KC];
#pragma unroll
        for (int h = h0; h < h0 + KH; ++h) {
#pragma unroll
          for (int c = 0; c < KC; ++c) {
            const float scale = __uint_as_float(K.s[h][D == 256 ? c >> 2 : 0] << 23);
#pragma unroll
            for (int p = 0; p < 4; ++p) kf[h - h0][c].w[p] = widen_byte(K.c[h][c], scale, p);
          }
          if (any_kbad) {   // a NaN block, or a page that does not exist
            keep_branch();
#pragma unroll
            for (int c = 0; c < KC; ++c) {
              const bool bad = at.lost[h] || K.s[h][D == 256 ? c >> 2 : 0] > kTopScale;
#pragma unroll
              for (int p = 0; p < 4; ++p) kf[h - h0][c].w[p] = bad ? 0x7FC07FC0u : kf[h - h0][c].w[p];
            }
          }
        }
        // read again for every tile: held across them they would take RT * D / 8 registers
        if constexpr (QL) asm volatile("" : "+v"(q_at));
        constexpr int RB = KH == 2 ? 1 : RT;   // row tiles whose fragments are read together
#pragma unroll
        for (int r0t = 0; r0t < RT; r0t += RB)
#pragma unroll
          for (int c = 0; c < KC; ++c) {
            Frag qf[RB];
#pragma unroll
            for (int x = 0; x < RB; ++x) qf[x] = QL ? q_lds[((r0t + x) * KC + c) * 64 + q_at] : q[QL ? 0 : r0t + x][c];
#pragma unroll
            for (int x = 0; x < RB; ++x)
#pragma unroll
              for (int h = h0; h < h0 + KH; ++h) {
                f32x4_t& d = s[r0t + x][h];
                if (c == 0) d = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
                d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf[h - h0][c].get(), qf[x].get(), d, 0, 0, 0);
              }
          }
      }
      if constexpr (LATE) load_v<D>(V, vc, vs, at, offs);
      at = place_of<D>(a, ahead, tok + kStep, last16);
      load_k<D>(K, kc, ks, at, offs);
      // after the reads of the queries: a wait for LDS counts scalar loads too, and waits for all
      ahead = find_pages(a, table, tok + 2 * kStep, last16);
      const bool edge = tok < lo_all || tok + 32 > min(hi_all, end);
      if (edge) {
        keep_branch();
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          int lo, hi;
          limits(rt, &lo, &hi);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int t = tok + 4 * g + 16 * (j >> 2) + (j & 3);
            if (!(t >= lo && t < min(hi, end))) s[rt][j >> 2][j & 3] = -__builtin_inff();
          }
        }
      }
      Frag pf[RT];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = s[rt][j >> 2][j & 3];
        // the lane's own largest score decides; the row's, over its four lanes, is needed when it moves
        const float top = max3(max3(f[0], f[1], f[2]), max3(f[3], f[4], f[5]), max3(f[6], f[7], f[7]));
        if (__builtin_amdgcn_ballot_w64(__builtin_fmaf(top, a.scale_log2, -run_m[rt]) > kSlack) != 0) {
          keep_branch();
          const float nm = max3(run_m[rt], row_max(top) * a.scale_log2, run_m[rt]);
          const float alpha = __builtin_amdgcn_exp2f(run_m[rt] - nm);
          run_m[rt] = nm;
          acc_l[rt] *= alpha;
#pragma unroll
          for (int cb = 0; cb < CB; ++cb) acc[rt][cb] *= alpha;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(f[j], a.scale_log2, -run_m[rt]));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const f32x2_t two = {f[2 * j], f[2 * j + 1]};
          pf[rt].w[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(two, bf16x2_t));
        }
      }

      // V scales of the lane's eight tokens
      const int shift = 8 * (D == 64 ? m >> 3 : D == 128 ? m >> 2 : (m >> 1) & 3);
      uint32_t byte[8];
      uint32_t top_vs = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        byte[j] = __builtin_amdgcn_ubfe(V.s[j >> 2][j & 3], shift, 8);
        top_vs = max(top_vs, byte[j]);
      }
      if (tok + 32 > seq.len) {   // behind the end of the sequence lies whatever the page held
        keep_branch();
        top_vs = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          if (tok + 16 * (j >> 2) + 4 * g + (j & 3) >= seq.len) byte[j] = 0;
          top_vs = max(top_vs, byte[j]);
        }
      }
      if (__builtin_amdgcn_ballot_w64(top_vs > kTopScale) != 0) {
        keep_branch();
        // NaN blocks among the values. A masked probability is 0 and 0 * NaN
        // would reach rows that do not see the token, so such blocks enter
        // the product as zeros, and the rows that see them are marked.
        // Lane 16 G + M holds token 16h + 4G + j, channels M * D/16 and on;
        // the outputs of lane (m, g) lie in the channels of M = 4g .. 4g+3.
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          int lo, hi;
          limits(rt, &lo, &hi);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint64_t who = __builtin_amdgcn_ballot_w64(byte[j] > kTopScale);
            if (who == 0) continue;
            for (int G = 0; G < 4; ++G) {
              const int t = tok + 16 * (j >> 2) + 4 * G + (j & 3);
#pragma unroll
              for (int x = 0; x < NP; ++x)
                if (t >= lo && t < min(hi, end) && (who >> (16 * G + 4 * g + 2 * x) & 1)) poison |= 1u << (rt * NP + x);
            }
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const bool bad = byte[j] > kTopScale;
          byte[j] = bad ? 127 : byte[j];
#pragma unroll
          for (int x = 0; x < VTile<D>::W; ++x) V.c[j >> 2][j & 3][x] = bad ? 0u : V.c[j >> 2][j & 3][x];
        }
      }

      // out += V^T P^T: two 16-channel blocks per byte of codes
#pragma unroll
      for (int p = 0; p < CB / 2; ++p) {
        Frag even, odd;
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
          const uint32_t x = widen_byte(V.c[j >> 2][j & 3][p >> 2], __uint_as_float(byte[j] << 23), p & 3);
          const uint32_t y = widen_byte(V.c[j >> 2][(j & 3) + 1][p >> 2], __uint_as_float(byte[j + 1] << 23), p & 3);
          even.w[j / 2] = __builtin_amdgcn_perm(y, x, 0x05040100u);
          odd.w[j / 2] = __builtin_amdgcn_perm(y, x, 0x07060302u);
        }
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          acc[rt][2 * p] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(even.get(), pf[rt].get(), acc[rt][2 * p], 0, 0, 0);
          acc[rt][2 * p + 1] =
              __builtin_amdgcn_mfma_f32_16x16x32_bf16(odd.get(), pf[rt].get(), acc[rt][2 * p + 1], 0, 0, 0);
        }
      }
      // a row of ones for V^T: the probabilities' sums
      const Frag ones = {{0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u}};
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
        acc_l[rt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones.get(), pf[rt].get(), acc_l[rt], 0, 0, 0);
      if (!LATE) load_v<D>(V, vc, vs, at, offs);
    };

    for (int ch = split; ch < sp.chunks; ch += a.splits) {
      const int begin = sp.first + ch * a.chunk;
      const int end = min(begin + a.chunk, sp.hi);
      int tok = begin + 32 * wave;
      if (tok >= end) continue;
      last16 = (end - 1) & ~15;
      KTile<D> K;
      VTile<D> V;
      Place at = place_of<D>(a, find_pages(a, table, tok, last16), tok, last16);
      Pages ahead = find_pages(a, table, tok + kStep, last16);
      // in the order in which the loop issues and awaits them: its waits
      // count the loads behind the one they are for, and hold for both
      __builtin_amdgcn_sched_barrier(0);
      load_k<D>(K, kc, ks, at, offs);
      __builtin_amdgcn_sched_barrier(0);
      if (!LATE) load_v<D>(V, vc, vs, at, offs);
      __builtin_amdgcn_sched_barrier(0);
      for (; tok < end; tok += kStep) tile(K, V, at, ahead, tok, end);
    }

    // Join the four waves: one row tile at a time through LDS.
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const float sum = acc_l[rt][0];
      __syncthreads();   // the buffer's last readers are done
      if (g == 0) {
        red_m[wave * 16 + m] = run_m[rt];
        red_l[wave * 16 + m] = sum;
      }
      // lane (m, g) holds row m, channels (4g + i) * D/16 + cb
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const bool nan = poison >> (rt * NP + (NP > 1 ? i >> 1 : 0)) & 1;
#pragma unroll
        for (int cb = 0; cb < CB; cb += 4) {
          f32x4_t v = {acc[rt][cb][i], acc[rt][cb + 1][i], acc[rt][cb + 2][i], acc[rt][cb + 3][i]};
          if (nan) v = f32x4_t{__builtin_nanf(""), __builtin_nanf(""), __builtin_nanf(""), __builtin_nanf("")};
          *reinterpret_cast<f32x4_t*>(&red[(wave * 16 + m) * LD + (4 * g + i) * CB + cb]) = v;
        }
      }
      __syncthreads();
      const int row = threadIdx.x >> 4;                 // 16 threads per row
      const int col = (threadIdx.x & 15) * (D / 16);    // D/16 channels each
      const int r = r0 + rt * 16 + row;
      float top = kNothing;
      float w[kWaves], l = 0.0f;
#pragma unroll
      for (int x = 0; x < kWaves; ++x) top = __builtin_fmaxf(top, red_m[x * 16 + row]);
#pragma unroll
      for (int x = 0; x < kWaves; ++x) {
        w[x] = __builtin_amdgcn_exp2f(red_m[x * 16 + row] - top);   // a NaN sum passes through any weight
        l += w[x] * red_l[x * 16 + row];
      }
      float o[D / 16];
#pragma unroll
      for (int e = 0; e < D / 16; ++e) {
        o[e] = 0.0f;
#pragma unroll
        for (int x = 0; x < kWaves; ++x) o[e] += w[x] * red[(x * 16 + row) * LD + col + e];
      }
      if (r < rows) {
        const int i = over(r, a.by_group);
        const int head = hk * a.group + (r - i * a.group);
        if (joined) {
          const int64_t at = ((int64_t)(seq.q0 + i) * heads_q + head) * a.splits + split;
#pragma unroll
          for (int e = 0; e < D / 16; e += 4)
            *reinterpret_cast<f32x4_t*>(a.part_o + at * D + col + e) = f32x4_t{o[e], o[e + 1], o[e + 2], o[e + 3]};
          if ((threadIdx.x & 15) == 0) *reinterpret_cast<f32x2_t*>(a.part_ml + at * 2) = f32x2_t{top, l};
        } else {
          const bool empty = see_hi(a, seq, i) <= see_lo(a, seq, i);      // a row that sees nothing is zero
          const float inv = 1.0f / l;
          char* p = static_cast<char*>(a.out) + ((int64_t)(seq.q0 + i) * a.ldo + (int64_t)head * D + col) * 2;
          uint32_t u[D / 32];
#pragma unroll
          for (int e = 0; e < D / 32; ++e) {
            const f32x2_t two = {empty ? 0.0f : o[2 * e] * inv, empty ? 0.0f : o[2 * e + 1] * inv};
            u[e] = __builtin_bit_cast(uint32_t, __builtin_convertvector(two, bf16x2_t));
          }
          if constexpr (D == 64) {
            *reinterpret_cast<u32x2_t*>(p) = u32x2_t{u[0], u[1]};
          } else {
#pragma unroll
            for (int e = 0; e < D / 32; e += 4)
              *reinterpret_cast<u32x4_t*>(p + 4 * e) = u32x4_t{u[e], u[e + 1], u[e + 2], u[e + 3]};
          }
        }
      }
    }
  }
}

// Joins the chunks of rows whose cache was split: a block per (query, head),
// D/4 threads across the row's columns, the rest along the chunks. The row's
// chunk count follows from the same arithmetic as in qknorm_attend; rows
// finished there are left alone. About 5 us as a launch of its own, mostly
// start-up and two round trips to memory (86 parts of 40 rows, 1.8 MB).
template <int D>
__global__ void __launch_bounds__(256) qknorm_attend_join(const AttendArgs a, int row_tile, int max_q) {
  constexpr int CT = D / 4;             // threads across
  constexpr int NG = 256 / CT;          // chunk groups
  __shared__ __align__(16) float red[NG * D];
  __shared__ float red_m[NG], red_l[NG];
  const int head = blockIdx.y;
  const int b = blockIdx.x / (uint32_t)max_q;
  const Sequence seq = sequence(a, b);
  const int heads_q = a.heads_k * a.group;
  const int grp = threadIdx.x / CT, col = (threadIdx.x & (CT - 1)) * 4;
  for (int i = blockIdx.x - b * max_q; i < seq.nq; i += max_q) {
    const int rows = seq.nq * a.group;
    const int in_group = head - (int)over(head, a.by_group) * a.group;
    const int r0 = (int)((uint32_t)(i * a.group + in_group) / (uint32_t)(16 * row_tile)) * (16 * row_tile);
    const Span sp = span(a, seq, over(r0, a.by_group), over(min(rows, r0 + 16 * row_tile) - 1, a.by_group));
    if (sp.chunks <= 1) continue;
    const int n = min(sp.chunks, a.splits);
    const int64_t at = ((int64_t)(seq.q0 + i) * heads_q + head) * a.splits;
    const float* ml = a.part_ml + at * 2;
    const float* po = a.part_o + at * D + col;
    float top = kNothing, l = 0.0f;
    f32x4_t o = {0.0f, 0.0f, 0.0f, 0.0f};
    // kAhead parts at a time, so that their loads are in flight together
    constexpr int kAhead = 4;
    for (int s0 = grp; s0 < n; s0 += kAhead * NG) {
      f32x2_t sum[kAhead];
      f32x4_t part[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int s = min(s0 + j * NG, n - 1);
        sum[j] = *reinterpret_cast<const f32x2_t*>(ml + 2 * s);
        part[j] = *reinterpret_cast<const f32x4_t*>(po + (int64_t)s * D);
      }
      float high = top;
#pragma unroll
      for (int j = 0; j < kAhead; ++j) high = __builtin_fmaxf(high, sum[j][0]);
      const float old = __builtin_amdgcn_exp2f(top - high);
      top = high;
      l *= old;
      o *= old;
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        if (s0 + j * NG >= n) break;
        const float w = __builtin_amdgcn_exp2f(sum[j][0] - top);
        l += w * sum[j][1];
        o += part[j] * w;
      }
    }
    __syncthreads();
    *reinterpret_cast<f32x4_t*>(&red[grp * D + col]) = o;
    if (col == 0) red_m[grp] = top, red_l[grp] = l;
    __syncthreads();
    if (grp == 0) {
      float all = kNothing;
#pragma unroll
      for (int x = 0; x < NG; ++x) all = __builtin_fmaxf(all, red_m[x]);
      l = 0.0f;
      o = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int x = 0; x < NG; ++x) {
        const float w = __builtin_amdgcn_exp2f(red_m[x] - all);
        l += w * red_l[x];
        o += *reinterpret_cast<const f32x4_t*>(&red[x * D + col]) * w;
      }
      const bool empty = see_hi(a, seq, i) <= see_lo(a, seq, i);
      const float inv = 1.0f / l;
      o = empty ? f32x4_t{0.0f, 0.0f, 0.0f, 0.0f} : o * inv;
      const f32x2_t x = {o[0], o[1]}, y = {o[2], o[3]};
      *reinterpret_cast<u32x2_t*>(static_cast<char*>(a.out) +
                                  ((int64_t)(seq.q0 + i) * a.ldo + (int64_t)head * D + col) * 2) =
          u32x2_t{__builtin_bit_cast(uint32_t, __builtin_convertvector(x, bf16x2_t)),
                  __builtin_bit_cast(uint32_t, __builtin_convertvector(y, bf16x2_t))};
    }
  }
}

template <int D>
void (*pick_attend(int rt))(const AttendArgs) {
  if (rt == 1) return qknorm_attend<D, 1>;
  if (rt == 2) return qknorm_attend<D, 2>;
  if constexpr (D < 256) {
    if (rt == 4) return qknorm_attend<D, 4>;
  }
  return nullptr;
}

}  // namespace

int launch_attend(const AttendPlan& p, const AttendArgs& args, void* stream, std::string* err) {
  void (*fn)(const AttendArgs) = p.head_dim == 64    ? pick_attend<64>(p.row_tile)
                                 : p.head_dim == 128 ? pick_attend<128>(p.row_tile)
                                                     : pick_attend<256>(p.row_tile);
  if (!fn) {
    *err = "no kernel compiled for this plan";
    return (int)hipErrorInvalidValue;
  }
  AttendArgs a = args;
  void* kargs[] = {&a};
  const int64_t grid = (int64_t)a.B * a.heads_k * a.row_tiles * a.splits;
  hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(fn), dim3((unsigned)grid), dim3(64 * kWaves), kargs, 0,
                                 static_cast<hipStream_t>(stream));
  if (e == hipSuccess && a.splits > 1) {
    int rt = p.row_tile;
    int mq = (int)p.max_q;
    void* jargs[] = {&a, &rt, &mq};
    const void* join = p.head_dim == 64    ? reinterpret_cast<const void*>(qknorm_attend_join<64>)
                       : p.head_dim == 128 ? reinterpret_cast<const void*>(qknorm_attend_join<128>)
                                           : reinterpret_cast<const void*>(qknorm_attend_join<256>);
    e = hipLaunchKernel(join, dim3((unsigned)(a.B * mq), (unsigned)(a.heads_k * a.group)), dim3(256), jargs, 0,
                        static_cast<hipStream_t>(stream));
  }
  if (e != hipSuccess) {
    *err = std::string("kernel launch: ") + hipGetErrorString(e);
    return (int)e;
  }
  return 0;
}

}  // namespace qkn

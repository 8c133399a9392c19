// Attention of new tokens over a paged key / value cache of bf16 rows or MXFP8
// (E4M3 codes, one E8M0 scale per 32 channels), on gfx950 (CDNA4).
//
// For query row r of a sequence and the cached tokens t it sees,
// out_r = sum_t softmax_t(scale q_r . k_t) v_t, in one pass over the cache:
// a running maximum m and sum l per row, and an accumulator that is rescaled
// when m grows. MXFP8 codes are widened to bf16 with their scale applied,
// exactly (four significant bits times a power of two, from 2^-130 on), so both products run on
// bf16 MFMA tiles with nothing lost on the K and V side. Probabilities are
// rounded to bf16, which the second product takes (at most half a step, 2^-8
// relative, averaged over the tokens); scores, m, l and the accumulator are
// float32, and l sums the rounded probabilities.
//
// Scores are formed transposed (tokens x rows), so that a lane holds one row's
// scores, and those are the positions it must hold of the second product's
// operand: probabilities go from one product to the other in registers. V passes
// through LDS, whose transposing reads give a lane eight tokens of one channel.
//
// Two kernels. qknorm_attend_few, for up to 32 rows of a sequence and key head:
// the four waves of a block take the 32-token tiles of its part of the cache in
// turn, K straight into registers, and join in LDS at the end. Bound by the
// cache's bytes: 64 single tokens of 40 over 8 heads of 128 on up to 8192 take 278 us
// from rows, 5.6 TB/s, and 153 from MXFP8, 5.3; one on 65536 in MXFP8 25 us and
// 5 us of joining its splits. Tiles of 32 tokens, since a wave's K and V in flight
// then fill its registers at two blocks a compute unit; two tiles in flight, and
// eight waves, were no faster.
//
// qknorm_attend_many, beyond: each wave takes 32 rows of its own, and all share K
// and V tiles of 64 tokens that the block stages in LDS, the next one loaded into
// registers behind the products. A wave of 32 rows reads each staged byte once for
// 32 x 32 x 16 products, half of what 16 rows would take of LDS; 64 tokens, so that
// two independent chains of products hide each other's latency. 4 x 531 .. 1024 rows
// of those heads on 4215 .. 8192 cached tokens: 370 us, 980 TFLOP/s (an 8192^3 library
// product reaches 1184), MXFP8 360. The matrix unit is busy 48 % and the vector unit,
// with the exponentials, roundings and maxima, 41 % of the time; without the loads it
// would take 337 us, without the exponentials 343.

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <string>

#include "qknorm_attend_device.hpp"

namespace qkn {
namespace {

typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));

constexpr int kWaves = 4;
constexpr uint32_t kTopScale8 = 246;      // largest scale byte of a finite MXFP8 block; above it, NaN
constexpr uint32_t kNaNs = 0x7FC07FC0u;   // two bf16 NaNs

// Formats of the cache. A lane moves 16 bytes at a time: kVW elements.
struct Rows16 {
  static constexpr bool kCodes = false;
  static constexpr int kVW = 8;
};
struct Mxfp8 {
  static constexpr bool kCodes = true;
  static constexpr int kVW = 16;
};

struct Raw {              // 16 bytes of a token's head, and their scale
  uint32_t w[4];
  uint32_t scale;
};

// Eight codes, two words, as bf16. (The conversion takes the scale's exponent field: 0 is 2^-127.)
__device__ __forceinline__ void widen8(const uint32_t* c, uint32_t scale_byte, uint32_t (&o)[4]) {
  const float s = __uint_as_float(scale_byte << 23);
  o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[0], s, false));
  o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[0], s, true));
  o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[1], s, false));
  o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[1], s, true));
}

// The elements of a lane's 16 bytes as bf16 words.
template <class F>
struct Piece16 {
  static constexpr int W = F::kVW / 2;
  uint32_t w[W];
  __device__ __forceinline__ void widen(const Raw& r) {
    if constexpr (F::kCodes) {
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        uint32_t o[4];
        widen8(r.w + 2 * p, r.scale, o);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[4 * p + i] = o[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = r.w[i];
    }
  }
  __device__ __forceinline__ void fill(uint32_t v) {
#pragma unroll
    for (int i = 0; i < W; ++i) w[i] = v;
  }
  // An infinity or NaN among the elements: an exponent of ones.
  __device__ __forceinline__ bool unusual() const {
    bool any = false;
#pragma unroll
    for (int i = 0; i < W; ++i) any = any || (w[i] & 0x7F80u) == 0x7F80u || (w[i] & 0x7F800000u) == 0x7F800000u;
    return any;
  }
  __device__ __forceinline__ void drop_unusual() {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      if ((w[i] & 0x7F80u) == 0x7F80u) w[i] &= 0xFFFF0000u;
      if ((w[i] & 0x7F800000u) == 0x7F800000u) w[i] &= 0xFFFFu;
    }
  }
  __device__ __forceinline__ void to_lds(char* p) const {
#pragma unroll
    for (int i = 0; i < W; i += 4)
      *reinterpret_cast<u32x4_t*>(p + 4 * i) = u32x4_t{w[i], w[i + 1], w[i + 2], w[i + 3]};
  }
};

template <class T>
__device__ __forceinline__ T load_at(uint64_t base, uint32_t offset) {
  typedef const T __attribute__((address_space(1)))* gptr;
  return *reinterpret_cast<gptr>(base + (uint64_t)offset);
}

// Of one of K and V, a key head of it: addresses in scalar registers.
struct Source {
  uint64_t rows, scales;
};

// A group of up to 16 tokens that lie in one page: where it begins. Tokens past
// the end of the chunk read its last 16 again, masked later.
struct Group {
  uint64_t rows, scales;
  bool lost;               // the page does not exist
};
template <int D>
__device__ __forceinline__ Group group_at(const AttendArgs& a, int page_id, int tok, int last16) {
  Group p;
  const int off = (tok <= (last16 | 15) ? tok : last16 | (tok & 15)) & ((1 << a.log2_page) - 1);
  p.lost = (uint32_t)page_id >= a.n_pages;
  const uint32_t page = p.lost ? 0 : page_id;
  p.rows = uniform64(page * (uint64_t)a.page_stride + (uint32_t)off * (uint64_t)a.token_stride);
  p.scales = uniform64(page * (uint64_t)a.scale_page_stride + (uint32_t)off * (uint64_t)(D / 32));
  return p;
}
__device__ __forceinline__ int page_of(const AttendArgs& a, const int32_t* table, int tok, int last16) {
  return load_uniform(table + (min(tok, last16) >> a.log2_page));
}

// Element (token, channel) of V as float32. For the few tiles with infinities or NaN
// next to a mask: what matters is whether it is one of them (the scale byte 0 may be 0 here).
template <class F>
__device__ __forceinline__ float value_at(const AttendArgs& a, const Source& v, const int32_t* table, int t, int channel) {
  const int id = load_uniform(table + (t >> a.log2_page));
  if ((uint32_t)id >= a.n_pages) return 0.0f;      // K's NaN makes the row NaN
  const uint64_t off = (uint32_t)(t & ((1 << a.log2_page) - 1));
  const uint64_t row = v.rows + (uint32_t)id * (uint64_t)a.page_stride + off * (uint64_t)a.token_stride;
  if constexpr (F::kCodes) {
    const uint32_t code = load_at<uint8_t>(row, channel);
    const uint32_t scale =
        load_at<uint8_t>(v.scales + (uint32_t)id * (uint64_t)a.scale_page_stride + off * (uint64_t)a.scale_row, channel >> 5);
    if (scale > kTopScale8) return __builtin_nanf("");
    return __builtin_amdgcn_cvt_f32_fp8(code, 0) * __uint_as_float(scale << 23);
  } else {
    return __uint_as_float((uint32_t)load_at<uint16_t>(row, 2 * channel) << 16);
  }
}

// Infinities and NaN among the values of tokens that some rows of a block see and
// others do not: 0 * NaN would reach the latter, so such elements enter the product
// as zeros where a tile of TOK tokens is at an edge, and are added here, at the end
// and where there were any, to a row that sees the tokens in [lo, hi): N of its
// channels. block_lo, block_hi: what every row sees, which tells the tiles apart.
template <class F, int TOK, int N>
__device__ __forceinline__ void add_unusual(const AttendArgs& a, const Source& v, const int32_t* table, const Span& sp,
                                            int split, int block_lo, int block_hi, int lo, int hi, int channel,
                                            float (&o)[N]) {
#pragma unroll 1
  for (int ch = split; ch < sp.chunks; ch += a.splits) {
    const int begin = sp.first + ch * a.chunk, end = min(begin + a.chunk, sp.hi);
#pragma unroll 1
    for (int tok = begin; tok < end; tok += TOK) {
      if (!(tok < block_lo || tok + TOK > min(block_hi, end))) continue;
#pragma unroll 1
      for (int t = tok; t < min(tok + TOK, end); ++t)
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float x = value_at<F>(a, v, table, t, channel + e);
          if (t >= lo && t < hi && !__builtin_isfinite(x)) o[e] += x;
        }
    }
  }
}

__device__ __forceinline__ s16x4_t read_transposed(const char* lds) {
  typedef __attribute__((address_space(3))) s16x4_t* lptr;
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lptr)(lds));
}
__device__ __forceinline__ Frag join4(s16x4_t lo, s16x4_t hi) {
  const u32x2_t a = __builtin_bit_cast(u32x2_t, lo), b = __builtin_bit_cast(u32x2_t, hi);
  return Frag{{a.x, a.y, b.x, b.y}};
}

__device__ __forceinline__ uint32_t pack2(float x, float y) {
  const f32x2_t two = {x, y};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(two, bf16x2_t));
}

// The running sum of a row's rounded probabilities (this lane's tokens).
__device__ __forceinline__ float add_pair(uint32_t w, float sum) {
  const uint32_t ones = 0x3F803F80u;
  return __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, w), __builtin_bit_cast(bf16x2_t, ones), sum, false);
}

// ------------------------------------------------------------------ few rows
// RT tiles of 16 rows; rows are query-major, all heads of a group side by side, so
// a decoded token's group shares one read of the cache.
template <class F, int D, int RT>
__global__ void __launch_bounds__(64 * kWaves, D == 256 ? 1 : 2) qknorm_attend_few(const AttendArgs a) {
  constexpr int CB = D / 16;                 // 16-channel blocks of the output
  constexpr int KC = D / 32;                 // 8-channel chunks a lane holds of a row
  constexpr int KL = F::kCodes ? KC / 2 : KC;         // 16-byte loads a lane makes of a K half
  constexpr int kPer = D / F::kVW;           // lanes across a token's V
  constexpr int kAt = 64 / kPer;             // tokens of one V load
  constexpr int VL = 32 / kAt;               // V loads of a tile
  constexpr int LDV = D * 2 + 32;            // bytes of a V row in LDS: four rows' 32-byte parts lie in distinct banks
  constexpr int LD = D + 4;                  // padded row of the join buffer
  constexpr int kStep = 32 * kWaves;
  constexpr int kTile = 32 * LDV, kJoin = 16 * LD * 4;      // bytes a wave
  __shared__ __align__(16) char lds[kWaves * (kTile > kJoin ? kTile : kJoin)];
  __shared__ float red_m[kWaves * 16], red_l[kWaves * 16];
  __shared__ int unusual;                    // some tile at an edge held infinities or NaN
  float* red = reinterpret_cast<float*>(lds);

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
  const Source ksrc{uniform64((uint64_t)a.cache[0] + hk * a.head_stride), uniform64((uint64_t)a.scales[0] + hk * a.scale_head_stride)};
  const Source vsrc{uniform64((uint64_t)a.cache[1] + hk * a.head_stride), uniform64((uint64_t)a.scales[1] + hk * a.scale_head_stride)};
  const int rows = seq.nq * a.group;
  const int heads_q = a.heads_k * a.group;
  char* vbuf = lds + wave * kTile;

  // K: token m of each half; rows: channels 32c + 8g and on of chunk c; codes:
  // 64c + 16g and on, two chunks a load
  const uint32_t k_off = m * (uint32_t)a.token_stride + g * 16;
  const uint32_t ks_off = m * (D / 32) + (g >> 1);
  const uint32_t v_off = (lane / kPer) * (uint32_t)a.token_stride + (lane % kPer) * 16;
  const uint32_t vs_off = (lane / kPer) * (D / 32) + (lane % kPer) / 2;
  const auto k_channel = [&](int c) { return F::kCodes ? 64 * (c >> 1) + 16 * g + 8 * (c & 1) : 32 * c + 8 * g; };

  for (int r0 = grid_tile * (16 * RT); r0 < rows; r0 += a.row_tiles * (16 * RT)) {
    const int i_first = over(r0, a.by_group);
    const int i_last = over(min(rows, r0 + 16 * RT) - 1, a.by_group);
    const Span sp = span(a, seq, i_first, i_last);
    const int lo_all = see_lo(a, seq, i_last), hi_all = see_hi(a, seq, i_first);   // every row sees these
    const bool joined = sp.chunks > 1 && a.splits > 1;   // partial results: the join finishes
    if (split > 0 && split >= sp.chunks) continue;       // nothing of the cache left for this block

    // This lane's row of each tile is m. What it sees is needed at the edges
    // alone and formed there.
    const auto limits = [&](int rt, int* lo, int* hi) {
      const int r = r0 + rt * 16 + m;
      const int i = r < rows ? (int)over(r, a.by_group) : 0;
      *lo = see_lo(a, seq, i);
      *hi = r < rows ? see_hi(a, seq, i) : 0;
    };
    Frag q[RT][KC];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int r = r0 + rt * 16 + m;
      const bool on = r < rows;
      const int i = on ? (int)over(r, a.by_group) : 0;
      const int head = hk * a.group + (on ? r - i * a.group : 0);
      const char* p = static_cast<const char*>(a.q) + ((int64_t)(seq.q0 + i) * a.ldq + (int64_t)head * D) * 2;
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        u32x4_t w = {0, 0, 0, 0};
        if (on) w = *reinterpret_cast<const u32x4_t*>(p + k_channel(c) * 2);
        q[rt][c] = Frag{{w.x, w.y, w.z, w.w}};
      }
    }
    if (threadIdx.x == 0) unusual = 0;
    __syncthreads();
    float run_m[RT], run_l[RT];
    f32x4_t acc[RT][CB];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      run_m[rt] = kNothing;
      run_l[rt] = 0.0f;
#pragma unroll
      for (int cb = 0; cb < CB; ++cb) acc[rt][cb] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    }

    for (int ch = split; ch < sp.chunks; ch += a.splits) {
      const int begin = sp.first + ch * a.chunk;
      const int end = min(begin + a.chunk, sp.hi);
      int tok = begin + 32 * wave;
      if (tok >= end) continue;
      const int last16 = (end - 1) & ~15;
      Raw K[2][KL], V[VL];
      const auto load_k = [&](const Group (&at)[2]) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int c = 0; c < KL; ++c) {
            const u32x4_t w = load_at<u32x4_t>(ksrc.rows + at[h].rows, k_off + 64 * c);
            K[h][c].w[0] = w.x, K[h][c].w[1] = w.y, K[h][c].w[2] = w.z, K[h][c].w[3] = w.w;
            if constexpr (F::kCodes) K[h][c].scale = load_at<uint8_t>(ksrc.scales + at[h].scales, ks_off + 2 * c);
          }
      };
      const auto load_v = [&](const Group (&at)[2]) {
#pragma unroll
        for (int i = 0; i < VL; ++i) {
          const int t0 = i * kAt;                        // first token of the load; VL of them may share a half
          const Group& h = at[t0 >> 4];
          const uint32_t in = (t0 & 15);
          const u32x4_t w = load_at<u32x4_t>(vsrc.rows + h.rows + in * (uint64_t)a.token_stride, v_off);
          V[i].w[0] = w.x, V[i].w[1] = w.y, V[i].w[2] = w.z, V[i].w[3] = w.w;
          if constexpr (F::kCodes) V[i].scale = load_at<uint8_t>(vsrc.scales + h.scales + in * (D / 32), vs_off);
        }
      };
      const auto groups = [&](const int (&id)[2], int t, Group (&at)[2]) {
#pragma unroll
        for (int h = 0; h < 2; ++h) at[h] = group_at<D>(a, id[h], t + 16 * h, last16);
      };
      const auto pages = [&](int t, int (&id)[2]) {
#pragma unroll
        for (int h = 0; h < 2; ++h) id[h] = page_of(a, table, t + 16 * h, last16);
      };
      Group at[2];
      int ahead[2];
      pages(tok, ahead);
      groups(ahead, tok, at);
      pages(tok + kStep, ahead);
      load_k(at);
      load_v(at);
      for (; tok < end; tok += kStep) {
        // scores, transposed: lane (m, g) gets tokens 16h + 4g + i of row m
        f32x4_t s[RT][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          Frag kf[KC];
          uint32_t top = 0;
          if constexpr (F::kCodes) {
#pragma unroll
            for (int c = 0; c < KL; ++c) {
              widen8(K[h][c].w, K[h][c].scale, kf[2 * c].w);
              widen8(K[h][c].w + 2, K[h][c].scale, kf[2 * c + 1].w);
              top = max(top, K[h][c].scale);
            }
          } else {
#pragma unroll
            for (int c = 0; c < KC; ++c)
#pragma unroll
              for (int p = 0; p < 4; ++p) kf[c].w[p] = K[h][c].w[p];
          }
          if (at[h].lost || (F::kCodes && __builtin_amdgcn_ballot_w64(top > kTopScale8) != 0)) {
            keep_branch();      // a page that does not exist, or a NaN block
#pragma unroll
            for (int c = 0; c < KC; ++c) {
              const bool bad = at[h].lost || (F::kCodes && K[h][F::kCodes ? c / 2 : c].scale > kTopScale8);
#pragma unroll
              for (int p = 0; p < 4; ++p) kf[c].w[p] = bad ? kNaNs : kf[c].w[p];
            }
          }
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            s[rt][h] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int c = 0; c < KC; ++c)
              s[rt][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf[c].get(), q[rt][c].get(), s[rt][h], 0, 0, 0);
          }
        }
        // V into LDS; its registers and K's are free for the wave's next tile
        const bool edge = tok < lo_all || tok + 32 > min(hi_all, end);
#pragma unroll
        for (int i = 0; i < VL; ++i) {
          const int row = i * kAt + lane / kPer;
          Piece16<F> p;
          p.widen(V[i]);
          const bool lost = at[(i * kAt) >> 4].lost;
          if (F::kCodes && __builtin_amdgcn_ballot_w64(V[i].scale > kTopScale8) != 0) {
            keep_branch();
            if (V[i].scale > kTopScale8) p.fill(kNaNs);
          }
          if (edge || lost) {
            keep_branch();
            // behind the end of the sequence lies whatever the page held
            if (lost || tok + row >= seq.len) p.fill(0);
            if (__builtin_amdgcn_ballot_w64(p.unusual()) != 0) {
              p.drop_unusual();
              if (lane == 0) unusual = 1;
            }
          }
          p.to_lds(vbuf + row * LDV + (lane % kPer) * (F::kVW * 2));
        }
        groups(ahead, tok + kStep, at);
        load_k(at);
        load_v(at);
        pages(tok + 2 * kStep, ahead);
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
            run_l[rt] *= alpha;
#pragma unroll
            for (int cb = 0; cb < CB; ++cb) acc[rt][cb] *= alpha;
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) f[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(f[j], a.scale_log2, -run_m[rt]));
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            pf[rt].w[j] = pack2(f[2 * j], f[2 * j + 1]);
            run_l[rt] = add_pair(pf[rt].w[j], run_l[rt]);
          }
        }
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        // out += V^T P^T. A transposing read gives lane (m, g) tokens 4g .. 4g + 3 of channel m
#pragma unroll
        for (int cb = 0; cb < CB; ++cb) {
          const char* p = vbuf + (4 * g + (m >> 2)) * LDV + (16 * cb + 4 * (m & 3)) * 2;
          const Frag vf = join4(read_transposed(p), read_transposed(p + 16 * LDV));
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
            acc[rt][cb] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf.get(), pf[rt].get(), acc[rt][cb], 0, 0, 0);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        __builtin_amdgcn_wave_barrier();
      }
    }

    // Join the four waves: one row tile at a time through LDS.
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      float sum = run_l[rt];       // of the lane's tokens: the row's is over its four lanes
      sum = swap_add16(sum);
      sum = swap_add32(sum);
      __syncthreads();   // the buffer's last readers are done
      if (g == 0) {
        red_m[wave * 16 + m] = run_m[rt];
        red_l[wave * 16 + m] = sum;
      }
      // lane (m, g) holds row m, channels 16 cb + 4g and on
#pragma unroll
      for (int cb = 0; cb < CB; ++cb)
        *reinterpret_cast<f32x4_t*>(&red[(wave * 16 + m) * LD + 16 * cb + 4 * g]) = acc[rt][cb];
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
        if (unusual) {
          keep_branch();
          add_unusual<F, 32>(a, vsrc, table, sp, split, lo_all, hi_all, see_lo(a, seq, i), see_hi(a, seq, i), col, o);
        }
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
          for (int e = 0; e < D / 32; ++e)
            u[e] = empty ? 0u : pack2(o[2 * e] * inv, o[2 * e + 1] * inv);
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
    __syncthreads();   // V tiles share the join buffer
  }
}

// ----------------------------------------------------------------- many rows
// A block's sequence, key head, tile of rows (kBlock) and split of the cache. Blocks
// take different times (a sequence's length, a row's place in it) and are more than
// the chip holds at once, so the longest go first: up to 64 sequences by their
// cached tokens, each one's last rows first, and blocks for rows that a sequence
// does not have come last of all. 4 x 531 .. 1024 rows on 4215 .. 8192 tokens, 40
// over 8 heads of 128, four waves a block: in the order of the sequences 680 us, so
// ordered and with both halves of a tile in flight 432; the order alone takes a
// simulated schedule from 1.37 to 1.04 of the mean load.
// Consecutive blocks take the key heads in turn: where they divide by 8, a head's
// blocks run on one XCD, whose L2 then holds its cache.
struct Work {
  int b, hk, tile, split;
};
__device__ __forceinline__ Work work_of(const AttendArgs& a, int block_rows) {
  Work w;
  if (a.B > 64) {
    const uint32_t rest = over(blockIdx.x, a.by_pairs);
    const uint32_t pair = blockIdx.x - rest * a.by_pairs.d;
    const uint32_t rev = over(rest, a.by_splits);
    w.split = rest - rev * a.by_splits.d;
    w.tile = a.row_tiles - 1 - (int)rev;
    w.b = over(pair, a.by_heads);
    w.hk = pair - w.b * a.heads_k;
    return w;
  }
  const uint32_t rest = over(blockIdx.x, a.by_heads);
  w.hk = blockIdx.x - rest * a.by_heads.d;
  const uint32_t unit = over(rest, a.by_splits);
  w.split = rest - unit * a.by_splits.d;
  // lane b: a sequence's tiles, and those of the ones before it
  const int lane = threadIdx.x & 63;
  int tiles = 0, len = -1;
  if (lane < a.B) {
    const Sequence s = sequence(a, lane);
    len = s.len;
    tiles = min((s.nq * a.group + block_rows - 1) / block_rows, a.row_tiles);
  }
  int before = 0;
  for (int x = 0; x < a.B; ++x) {
    const int l = __builtin_amdgcn_readlane(len, x), n = __builtin_amdgcn_readlane(tiles, x);
    if (l > len || (l == len && x < lane)) before += n;
  }
  const uint64_t mine = __builtin_amdgcn_ballot_w64((int)unit >= before && (int)unit < before + tiles);
  if (mine == 0) {
    w.b = -1;
    return w;
  }
  w.b = __builtin_ctzll(mine);
  w.tile = __builtin_amdgcn_readlane(tiles, w.b) - 1 - ((int)unit - __builtin_amdgcn_readlane(before, w.b));
  return w;
}

// NW waves of 32 rows each. K and V tiles of kTok tokens in LDS, two of each:
// one is read while the next one, loaded into registers behind the products,
// waits to be written.
template <class F, int D, int NW>
__global__ void __launch_bounds__(64 * NW, D == 64 ? 3 : D == 128 ? 2 : 1) qknorm_attend_many(const AttendArgs a) {
  constexpr int TB = 2;                      // 32-token parts of a tile
  constexpr int kTok = 32 * TB;
  constexpr int MB = D / 32;                 // 32-channel blocks of the output
  constexpr int KS = D / 16;                 // steps of the first product
  constexpr int kPer = D / F::kVW;           // lanes across a token
  constexpr int kAt = 64 / kPer;             // tokens of one wave's load
  static_assert(kTok % (NW * kAt) == 0, "every wave loads the same share of a tile");
  constexpr int PL = kTok / (NW * kAt);      // loads a thread makes of K, and of V
  constexpr int LDK = D * 2 + 16, LDV = D * 2 + 64;   // bytes of a row: no two of those read together share a bank
  constexpr int kBlock = 32 * NW;   // rows of a block
  constexpr int kTileK = kTok * LDK, kTileV = kTok * LDV;
  constexpr int kOut = D < 128 ? D : 128;    // columns of the results on their way out at a time
  constexpr int LDO = kOut + 4;
  constexpr int kTiles = 2 * (kTileK + kTileV), kResults = NW * 32 * LDO * 4;
  __shared__ __align__(16) char lds[kTiles > kResults ? kTiles : kResults];
  char* const kbuf = lds;
  char* const vbuf = lds + 2 * kTileK;
  __shared__ int unusual;                    // some tile at an edge held infinities or NaN

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = lane & 31, g = lane >> 5;
  const Work at_work = work_of(a, kBlock);
  const int split = at_work.split, grid_tile = at_work.tile, b = at_work.b, hk = at_work.hk;
  if (b < 0) return;

  const Sequence seq = sequence(a, b);
  const int32_t* table = a.table + b * a.ld_table;
  const Source ksrc{uniform64((uint64_t)a.cache[0] + hk * a.head_stride), uniform64((uint64_t)a.scales[0] + hk * a.scale_head_stride)};
  const Source vsrc{uniform64((uint64_t)a.cache[1] + hk * a.head_stride), uniform64((uint64_t)a.scales[1] + hk * a.scale_head_stride)};
  const int rows = seq.nq * a.group;
  const int heads_q = a.heads_k * a.group;
  const uint32_t off = (lane / kPer) * (uint32_t)a.token_stride + (lane % kPer) * 16;
  const uint32_t s_off = (lane / kPer) * (D / 32) + (lane % kPer) / 2;

  for (int b0 = grid_tile * kBlock; b0 < rows; b0 += a.row_tiles * kBlock) {
    const int i_first = over(b0, a.by_group);
    const int i_last = over(min(rows, b0 + kBlock) - 1, a.by_group);
    const Span sp = span(a, seq, i_first, i_last);
    const bool joined = sp.chunks > 1 && a.splits > 1;
    if (split > 0 && split >= sp.chunks) continue;
    const int block_lo = see_lo(a, seq, i_last), block_hi = see_hi(a, seq, i_first);   // every row of the block sees these
    // this wave's rows: [r0, r1), what they see together and each
    const int r0 = b0 + wave * 32, r1 = min(rows, r0 + 32);
    const bool live = r0 < rows;
    const int w_first = live ? (int)over(r0, a.by_group) : 0, w_last = live ? (int)over(r1 - 1, a.by_group) : 0;
    const int any_lo = see_lo(a, seq, w_first), any_hi = live ? see_hi(a, seq, w_last) : 0;
    const int lo_all = see_lo(a, seq, w_last), hi_all = r1 - r0 == 32 ? see_hi(a, seq, w_first) : 0;

    const auto limits = [&](int* lo, int* hi) {
      const int r = r0 + m;
      const int i = r < rows ? (int)over(r, a.by_group) : 0;
      *lo = see_lo(a, seq, i);
      *hi = r < rows ? see_hi(a, seq, i) : 0;
    };
    Frag q[KS];
    {
      const int r = r0 + m;
      const bool on = r < rows;
      const int i = on ? (int)over(r, a.by_group) : 0;
      const int head = hk * a.group + (on ? r - i * a.group : 0);
      const char* p = static_cast<const char*>(a.q) + ((int64_t)(seq.q0 + i) * a.ldq + (int64_t)head * D) * 2;
#pragma unroll
      for (int c = 0; c < KS; ++c) {
        u32x4_t w = {0, 0, 0, 0};
        if (on) w = *reinterpret_cast<const u32x4_t*>(p + (16 * c + 8 * g) * 2);
        q[c] = Frag{{w.x, w.y, w.z, w.w}};
      }
    }
    if (threadIdx.x == 0) unusual = 0;
    float run_m = kNothing, run_l = 0.0f;
    f32x16_t acc[MB];
#pragma unroll
    for (int mb = 0; mb < MB; ++mb)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[mb][i] = 0.0f;

    for (int ch = split; ch < sp.chunks; ch += a.splits) {
      const int begin = sp.first + ch * a.chunk;
      const int end = min(begin + a.chunk, sp.hi);
      const int last16 = (end - 1) & ~15;
      Raw K[PL], V[PL];
      uint32_t lost = 0;               // bits of the loads whose page does not exist
      // page ids of the next 64 groups of 16 tokens, a lane's each: one load for 16
      // tiles, ahead of its use (a scalar lookup would hold up the tile's loads)
      const auto pages_from = [&](int tok) { return table[min(tok + 16 * lane, last16) >> a.log2_page]; };
      int ids = pages_from(begin), ids_from = begin, ids_next = pages_from(begin + 1024);
      // this wave's share of a tile: tokens (x * NW + wave) * kAt and on
      const auto load = [&](int tok) {
        if (tok >= ids_from + 1024) {
          ids_from += 1024;
          ids = ids_next;
          ids_next = pages_from(ids_from + 1024);
        }
        lost = 0;
#pragma unroll
        for (int x = 0; x < PL; ++x) {
          const int t = tok + (x * NW + wave) * kAt;
          const int id = __builtin_amdgcn_readlane(ids, (t - ids_from) >> 4);
          const Group at = group_at<D>(a, id, t, last16);
          lost |= (uint32_t)at.lost << x;
          const u32x4_t w = load_at<u32x4_t>(ksrc.rows + at.rows, off);
          K[x].w[0] = w.x, K[x].w[1] = w.y, K[x].w[2] = w.z, K[x].w[3] = w.w;
          const u32x4_t v = load_at<u32x4_t>(vsrc.rows + at.rows, off);
          V[x].w[0] = v.x, V[x].w[1] = v.y, V[x].w[2] = v.z, V[x].w[3] = v.w;
          if constexpr (F::kCodes) {
            K[x].scale = load_at<uint8_t>(ksrc.scales + at.scales, s_off);
            V[x].scale = load_at<uint8_t>(vsrc.scales + at.scales, s_off);
          }
        }
      };
      const int put_k = lane / kPer * LDK + lane % kPer * (F::kVW * 2), put_v = lane / kPer * LDV + lane % kPer * (F::kVW * 2);
      const auto store = [&](int tok, int buf) {
        const bool edge = tok < block_lo || tok + kTok > min(block_hi, end);
        uint32_t top = 0;
        if constexpr (F::kCodes) {
#pragma unroll
          for (int x = 0; x < PL; ++x) top = max(top, max(K[x].scale, V[x].scale));
        }
        char* const kd = kbuf + buf * kTileK + put_k;
        char* const vd = vbuf + buf * kTileV + put_v;
        if (edge || lost != 0 || (F::kCodes && __builtin_amdgcn_ballot_w64(top > kTopScale8) != 0)) {
          keep_branch();
#pragma unroll
          for (int x = 0; x < PL; ++x) {
            const int row = (x * NW + wave) * kAt;
            const bool gone = lost >> x & 1;
            Piece16<F> p;
            p.widen(K[x]);
            if (gone || (F::kCodes && K[x].scale > kTopScale8)) p.fill(kNaNs);
            p.to_lds(kd + row * LDK);
            p.widen(V[x]);
            if (F::kCodes && V[x].scale > kTopScale8) p.fill(kNaNs);
            // behind the end of the sequence lies whatever the page held
            if (gone || tok + row + lane / kPer >= seq.len) p.fill(0);
            if (edge && __builtin_amdgcn_ballot_w64(p.unusual()) != 0) {
              p.drop_unusual();
              if (lane == 0) unusual = 1;
            }
            p.to_lds(vd + row * LDV);
          }
        } else {
#pragma unroll
          for (int x = 0; x < PL; ++x) {
            const int row = (x * NW + wave) * kAt;
            Piece16<F> p;
            p.widen(K[x]);
            p.to_lds(kd + row * LDK);
            p.widen(V[x]);
            p.to_lds(vd + row * LDV);
          }
        }
      };
      int tok = begin, cur = 0;
      load(tok);
      __syncthreads();                 // the last chunk's readers are done
      store(tok, 0);
      __syncthreads();
      for (; tok < end; tok += kTok, cur ^= 1) {
        const bool more = tok + kTok < end;
        if (more) load(tok + kTok);
        if (tok < any_hi && tok + kTok > any_lo) {     // some row of this wave sees something
          const bool edge = tok < lo_all || tok + kTok > min(hi_all, end);
          // scores of both 32-token halves, transposed: lane (m, g) gets tokens
          // 32 tb + 8 (i / 4) + 4g + i % 4 of row m
          f32x16_t s[TB];
#pragma unroll
          for (int tb = 0; tb < TB; ++tb)
#pragma unroll
            for (int i = 0; i < 16; ++i) s[tb][i] = 0.0f;
          const char* kp = kbuf + cur * kTileK + m * LDK + g * 16;
          // reads of K ahead of the products that take them, which the compiler would
          // otherwise wait for two by two (two, three, six or eight ahead measure the same)
          constexpr int kAhead = 4;
          Frag kf[TB * KS];
          const auto read_k = [&](int i) {
            const u32x4_t w = *reinterpret_cast<const u32x4_t*>(kp + 32 * (i % TB) * LDK + 32 * (i / TB));
            kf[i] = Frag{{w.x, w.y, w.z, w.w}};
          };
#pragma unroll
          for (int i = 0; i < kAhead; ++i) read_k(i);
          __builtin_amdgcn_sched_group_barrier(0x100, kAhead, 0);   // LDS reads
#pragma unroll
          for (int i = 0; i < TB * KS; ++i) {
            if (i + kAhead < TB * KS) read_k(i + kAhead);
            s[i % TB] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf[i].get(), q[i / TB].get(), s[i % TB], 0, 0, 0);
            __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);        // a product
            if (i + kAhead < TB * KS) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
          }
          if (edge) {
            keep_branch();
            int lo, hi;
            limits(&lo, &hi);
#pragma unroll
            for (int tb = 0; tb < TB; ++tb)
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const int t = tok + 32 * tb + 8 * (i >> 2) + 4 * g + (i & 3);
                if (!(t >= lo && t < min(hi, end))) s[tb][i] = -__builtin_inff();
              }
          }
          // the lane's own largest score decides; the row's, over its two lanes, is needed when it moves
          float top = s[0][0];
#pragma unroll
          for (int i = 1; i < 16 * TB; i += 2)
            top = max3(top, s[i / 16][i % 16], s[(i + 1) / 16 % TB][(i + 1) % 16]);
          if (__builtin_amdgcn_ballot_w64(__builtin_fmaf(top, a.scale_log2, -run_m) > kSlack) != 0) {
            keep_branch();
            const auto o = __builtin_amdgcn_permlane32_swap(__float_as_uint(top), __float_as_uint(top), false, false);
            const float all = max3(__uint_as_float(o[0]), __uint_as_float(o[1]), __uint_as_float(o[1]));
            const float nm = max3(run_m, all * a.scale_log2, run_m);
            const float alpha = __builtin_amdgcn_exp2f(run_m - nm);
            run_m = nm;
            run_l *= alpha;
#pragma unroll
            for (int mb = 0; mb < MB; ++mb) acc[mb] *= alpha;
          }
          // This product goes before the other waves of its SIMD, whose exponentials and
          // conversions fill in between: 390 us at equal priority, 383 so, for 8192 tokens of
          // 32 heads on 8 of 128 channels, 16384 cached (381 and 373 with rows of MXFP8; the
          // first product's priority makes no difference)
          __builtin_amdgcn_s_setprio(1);
          // out += V^T P^T. A transposing read gives 16 lanes four tokens of 16 channels: lane
          // (m, g) holds tokens 4g .. 4g + 3 and 8 + 4g .. of channel m, as it holds of P
          const char* vp = vbuf + cur * kTileV + (4 * g + ((lane & 15) >> 2)) * LDV + (16 * ((lane >> 4) & 1) + 4 * (lane & 3)) * 2;
          // two reads ahead of the products and of the exponentials before them: heads of 256
          // take 483 us instead of 557, others 1 % less; four ahead, 503
          constexpr int kAheadV = 2;
          Frag vf[2 * TB * MB];
          const auto read_v = [&](int n) {
            const char* p = vp + 16 * (n / MB) * LDV + 64 * (n % MB);
            vf[n] = join4(read_transposed(p), read_transposed(p + 8 * LDV));
          };
#pragma unroll
          for (int n = 0; n < kAheadV; ++n) read_v(n);
#pragma unroll
          for (int ks = 0; ks < 2 * TB; ++ks) {
            Frag pf;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int i = 8 * (ks & 1) + 2 * j;
              const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(s[ks >> 1][i], a.scale_log2, -run_m));
              const float y = __builtin_amdgcn_exp2f(__builtin_fmaf(s[ks >> 1][i + 1], a.scale_log2, -run_m));
              pf.w[j] = pack2(x, y);
              run_l = add_pair(pf.w[j], run_l);
            }
#pragma unroll
            for (int mb = 0; mb < MB; ++mb) {
              const int n = ks * MB + mb;
              if (n + kAheadV < 2 * TB * MB) read_v(n + kAheadV);
              acc[mb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf[n].get(), pf.get(), acc[mb], 0, 0, 0);
            }
          }
          __builtin_amdgcn_s_setprio(0);
        }
        if (more) store(tok + kTok, cur ^ 1);
        __syncthreads();
      }
    }

    // Out through LDS, 32 rows of each wave at a time and at most 128 columns: lane (m, g)
    // holds row m, channels 32 mb + 8 (i / 4) + 4g + i % 4, and stores eight neighbouring
    // ones of a row.
    float* const res = reinterpret_cast<float*>(lds) + wave * 32 * LDO;
    constexpr int kAcross = kOut / 8;        // lanes across a row
#pragma unroll
    for (int mb0 = 0; mb0 < MB; mb0 += kOut / 32) {
      const float sum = swap_add32(run_l);
#pragma unroll
      for (int mb = 0; mb < kOut / 32; ++mb)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const f32x16_t& o = acc[mb0 + mb];
          *reinterpret_cast<f32x4_t*>(res + m * LDO + 32 * mb + 8 * x + 4 * g) =
              f32x4_t{o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]};
        }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
#pragma unroll 1
      for (int y = 0; y < 32; y += 64 / kAcross) {
        const int row = y + lane / kAcross, at = (lane % kAcross) * 8, col = 32 * mb0 + at;
        const int r = r0 + row;
        const float l = __shfl(sum, row), rm = __shfl(run_m, row);
        if (r >= rows) continue;
        float o[8];
#pragma unroll
        for (int e = 0; e < 8; e += 4) {
          const f32x4_t v = *reinterpret_cast<const f32x4_t*>(res + row * LDO + at + e);
          o[e] = v[0], o[e + 1] = v[1], o[e + 2] = v[2], o[e + 3] = v[3];
        }
        const int i = over(r, a.by_group);
        const int head = hk * a.group + (r - i * a.group);
        if (unusual) {
          keep_branch();
          add_unusual<F, kTok>(a, vsrc, table, sp, split, block_lo, block_hi, see_lo(a, seq, i), see_hi(a, seq, i), col, o);
        }
        if (joined) {
          const int64_t part_at = ((int64_t)(seq.q0 + i) * heads_q + head) * a.splits + split;
          float* p = a.part_o + part_at * D + col;
          *reinterpret_cast<f32x4_t*>(p) = f32x4_t{o[0], o[1], o[2], o[3]};
          *reinterpret_cast<f32x4_t*>(p + 4) = f32x4_t{o[4], o[5], o[6], o[7]};
          if (col == 0) *reinterpret_cast<f32x2_t*>(a.part_ml + part_at * 2) = f32x2_t{rm, l};
        } else {
          const bool empty = see_hi(a, seq, i) <= see_lo(a, seq, i);      // a row that sees nothing is zero
          const float inv = 1.0f / l;
          u32x4_t u = {pack2(o[0] * inv, o[1] * inv), pack2(o[2] * inv, o[3] * inv), pack2(o[4] * inv, o[5] * inv),
                       pack2(o[6] * inv, o[7] * inv)};
          if (empty) u = u32x4_t{0, 0, 0, 0};
          *reinterpret_cast<u32x4_t*>(static_cast<char*>(a.out) + ((int64_t)(seq.q0 + i) * a.ldo + (int64_t)head * D + col) * 2) = u;
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
    __syncthreads();     // the next rows' tiles, and `unusual`
  }
}

using AttendFn = void (*)(const AttendArgs);

template <class F, int D>
AttendFn pick_wide(int row_tile) {
  if (row_tile == 1) return qknorm_attend_few<F, D, 1>;
  if (row_tile == 2) return qknorm_attend_few<F, D, 2>;
  if (row_tile == 8) return qknorm_attend_many<F, D, 4>;
  if constexpr (D == 128) {
    if (row_tile == 16) return qknorm_attend_many<F, D, 8>;
  }
  return nullptr;
}

template <class F>
AttendFn pick_wide_width(const AttendPlan& p) {
  return p.head_dim == 64    ? pick_wide<F, 64>(p.row_tile)
         : p.head_dim == 128 ? pick_wide<F, 128>(p.row_tile)
                             : pick_wide<F, 256>(p.row_tile);
}

}  // namespace

int launch_attend_wide(bool mx8, const AttendPlan& p, const AttendArgs& args, void* stream, std::string* err) {
  const AttendFn fn = mx8 ? pick_wide_width<Mxfp8>(p) : pick_wide_width<Rows16>(p);
  if (!fn) {
    *err = "no kernel compiled for this plan";
    return (int)hipErrorInvalidValue;
  }
  AttendArgs a = args;
  void* kargs[] = {&a};
  const int64_t grid = (int64_t)a.B * a.heads_k * a.row_tiles * a.splits;
  const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(fn), dim3((unsigned)grid),
                                       dim3(p.row_tile == 16 ? 512 : 64 * kWaves),
                                       kargs, 0, static_cast<hipStream_t>(stream));
  if (e == hipSuccess && a.splits > 1) return launch_attend_join(p, a, stream, err);
  if (e != hipSuccess) {
    *err = std::string("kernel launch: ") + hipGetErrorString(e);
    return (int)e;
  }
  return 0;
}

}  // namespace qkn

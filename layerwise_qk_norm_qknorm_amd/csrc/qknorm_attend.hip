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
// (half a step, 2^-9 relative, averaged over the tokens), as large as the
// rounding of the output itself. Scores, m, l and the accumulator are
// float32.
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
// With one or two row tiles the cache's bytes bound it; with four (prompts)
// the vector unit does: widening, exponentials and masks cost about as much
// as the MFMA tiles take.

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

__device__ __forceinline__ float row_max(float v) {   // over the four lanes that hold a row
  auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __builtin_fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
  p = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __builtin_fmaxf(__uint_as_float(p[0]), __uint_as_float(p[1]));
}

// Codes and scales of one 32-token tile, as one lane holds them: lane = 16 g
// + m. K: token m of each half, a quarter of its channels (chosen by g). V:
// tokens 4g .. 4g+3 of each half, channels m * D/16 and on.
template <int D>
struct Tile {
  static constexpr int KW = D / 32;               // words of K codes per half
  static constexpr int KS = D == 256 ? 2 : 1;     // K scales per half
  static constexpr int VW = D == 256 ? 2 : 1;     // words of V codes per token
  uint32_t k[2][KW];
  uint32_t ks[2][KS];
  uint32_t v[2][4][VW];
  uint32_t vs[2][4];                              // V scale bytes
  bool lost[2];                                   // the page id was out of range
};

template <int D>
__device__ __forceinline__ void load_tile(Tile<D>& T, const AttendArgs& a, const int32_t* table, int64_t head_codes,
                                          int64_t head_scales, int64_t tok, int64_t last16, int lane) {
  const int m = lane & 15, g = lane >> 4;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    // past the end of the sequence: its last 16 tokens again, masked later
    int64_t t = tok + 16 * h;
    t = t < last16 ? t : last16;
    int page = table[t >> a.log2_page];
    T.lost[h] = page < 0 || page >= a.n_pages;
    page = T.lost[h] ? 0 : page;
    const int off = (int)(t & (((int64_t)1 << a.log2_page) - 1));
    const int64_t c0 = page * a.page_stride + head_codes + (int64_t)off * (D / 2);
    const int64_t s0 = page * a.scale_page_stride + head_scales + (int64_t)off * (D / 32);
    const uint8_t* kc = a.cache[0] + c0;
    const uint8_t* vc = a.cache[1] + c0;
    const uint8_t* ks = a.scales[0] + s0;
    const uint8_t* vs = a.scales[1] + s0;
    if constexpr (D == 64) {
      const u32x2_t w = __builtin_nontemporal_load(reinterpret_cast<const u32x2_t*>(kc + m * 32 + g * 8));
      T.k[h][0] = w.x, T.k[h][1] = w.y;
      T.ks[h][0] = ks[m * 2 + (g >> 1)];
    } else {
#pragma unroll
      for (int sp = 0; sp < D / 128; ++sp) {
        const u32x4_t w =
            __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(kc + m * (D / 2) + 64 * sp + g * 16));
        T.k[h][4 * sp] = w.x, T.k[h][4 * sp + 1] = w.y, T.k[h][4 * sp + 2] = w.z, T.k[h][4 * sp + 3] = w.w;
        T.ks[h][sp] = ks[m * (D / 32) + 4 * sp + g];
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint8_t* p = vc + (4 * g + j) * (D / 2) + m * (D / 32);
      if constexpr (D == 64) {
        T.v[h][j][0] = *reinterpret_cast<const uint16_t*>(p);
      } else if constexpr (D == 128) {
        T.v[h][j][0] = __builtin_nontemporal_load(reinterpret_cast<const uint32_t*>(p));
      } else {
        const u32x2_t w = __builtin_nontemporal_load(reinterpret_cast<const u32x2_t*>(p));
        T.v[h][j][0] = w.x, T.v[h][j][1] = w.y;
      }
    }
    // the scale words of the lane's four tokens; the byte is taken in use
    if constexpr (D == 64) {
      const u32x2_t w = *reinterpret_cast<const u32x2_t*>(vs + 8 * g);
      T.vs[h][0] = w.x, T.vs[h][1] = w.x >> 16, T.vs[h][2] = w.y, T.vs[h][3] = w.y >> 16;
    } else if constexpr (D == 128) {
      const u32x4_t w = *reinterpret_cast<const u32x4_t*>(vs + 16 * g);
      T.vs[h][0] = w.x, T.vs[h][1] = w.y, T.vs[h][2] = w.z, T.vs[h][3] = w.w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        T.vs[h][j] = *reinterpret_cast<const uint32_t*>(vs + (4 * g + j) * 8 + (m >> 3) * 4);
    }
  }
}

// The channel at which chunk c (8 channels) of lane group g begins.
template <int D>
__device__ __forceinline__ int k_channel(int g, int c) {
  return D == 64 ? 16 * g + 8 * c : 128 * (c >> 2) + 32 * g + 8 * (c & 3);
}

template <int D, int RT>
__global__ void __launch_bounds__(64 * kWaves, RT * D <= 256 ? 2 : 1) qknorm_attend(const AttendArgs a) {
  constexpr int CB = D / 16;                 // 16-channel blocks of the output
  constexpr int LD = D + 4;                  // padded row of the join buffer
  __shared__ __align__(16) float red[kWaves * 16 * LD];
  __shared__ float red_m[kWaves * 16], red_l[kWaves * 16];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m = lane & 15, g = lane >> 4;
  // blocks of one (sequence, key head) lie a multiple of their count apart:
  // on one XCD, whose L2 then holds that head's cache, where it divides by 8
  const uint32_t pairs = (uint32_t)a.B * a.heads_k;
  const uint32_t rest = blockIdx.x / pairs;
  const uint32_t pair = blockIdx.x - rest * pairs;
  const int split = rest % (uint32_t)a.splits;
  const int tile_of_grid = a.row_tiles - 1 - (int)(rest / (uint32_t)a.splits);   // long rows first
  const int b = pair / (uint32_t)a.heads_k;
  const int hk = pair - b * a.heads_k;

  int64_t q0 = b, nq = 1;
  if (a.cu_q) {
    q0 = a.cu_q[b];
    int64_t q1 = a.cu_q[b + 1];
    q0 = q0 < 0 ? 0 : q0 > a.T ? a.T : q0;
    q1 = q1 < q0 ? q0 : q1 > a.T ? a.T : q1;
    nq = q1 - q0;
  }
  int64_t len = a.seq_lens[b];
  len = len < 0 ? 0 : len > a.table_tokens ? a.table_tokens : len;
  const int64_t last16 = len > 0 ? (len - 1) & ~(int64_t)15 : 0;
  const int32_t* table = a.table + b * a.ld_table;
  const int64_t head_codes = hk * a.head_stride, head_scales = hk * a.scale_head_stride;
  const int64_t rows = nq * a.group;
  const int heads_q = a.heads_k * a.group;

  for (int64_t r0 = (int64_t)tile_of_grid * (16 * RT); r0 < rows; r0 += (int64_t)a.row_tiles * (16 * RT)) {
    // what the tile's rows see: tokens [lo, hi), all of them within [lo_all, hi_all)
    const int64_t i_first = r0 / a.group;
    const int64_t r_end = rows < r0 + 16 * RT ? rows : r0 + 16 * RT;
    const int64_t i_last = (r_end - 1) / a.group;
    const int64_t base = len - nq;           // position of query i: base + i
    const auto hi_of = [&](int64_t i) {
      const int64_t pos = base + i;
      return pos < 0 ? (int64_t)0 : a.causal ? pos + 1 : len;
    };
    const auto lo_of = [&](int64_t i) {
      const int64_t lo = base + i - a.window + 1;
      return a.window && lo > 0 ? lo : (int64_t)0;
    };
    const int64_t lo = lo_of(i_first), hi = hi_of(i_last);
    const int64_t lo_all = lo_of(i_last), hi_all = hi_of(i_first);
    const int64_t first = lo & ~(int64_t)31;           // tiles start at multiples of 32 tokens
    const int64_t chunks = hi > lo ? (hi - first + a.chunk - 1) / a.chunk : 0;
    const bool joined = chunks > 1 && a.splits > 1;    // partial results: qknorm_attend_join finishes
    if (split > 0 && split >= chunks) continue;        // nothing of the cache left for this block

    // row state: this lane's row of each tile is m
    int row_lo[RT], row_hi[RT];
    Frag q[RT][D / 32];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int64_t r = r0 + rt * 16 + m;
      const bool on = r < rows;
      const int64_t i = on ? r / a.group : 0;
      row_lo[rt] = on ? (int)(lo_of(i) - first < 0 ? 0 : lo_of(i) - first) : 0;
      row_hi[rt] = on ? (int)(hi_of(i) - first) : 0;
      const int head = hk * a.group + (int)(on ? r - i * a.group : 0);
      const char* p = static_cast<const char*>(a.q) + ((q0 + i) * a.ldq + (int64_t)head * D) * 2;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        u32x4_t w = {0, 0, 0, 0};
        if (on) w = *reinterpret_cast<const u32x4_t*>(p + k_channel<D>(g, c) * 2);
        q[rt][c].w[0] = w.x, q[rt][c].w[1] = w.y, q[rt][c].w[2] = w.z, q[rt][c].w[3] = w.w;
      }
    }
    float run_m[RT], run_l[RT];
    f32x4_t acc[RT][CB];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      run_m[rt] = -__builtin_inff();
      run_l[rt] = 0.0f;
#pragma unroll
      for (int cb = 0; cb < CB; ++cb) acc[rt][cb] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    }

    for (int64_t ch = split; ch < chunks; ch += a.splits) {
      const int64_t begin = first + ch * a.chunk;
      const int64_t end = begin + a.chunk < hi ? begin + a.chunk : hi;
      Tile<D> next;
      int64_t tok = begin + 32 * wave;
      if (tok < end) load_tile<D>(next, a, table, head_codes, head_scales, tok, last16, lane);
      for (; tok < end; tok += 32 * kWaves) {
        Tile<D> T = next;
        if (tok + 32 * kWaves < end)
          load_tile<D>(next, a, table, head_codes, head_scales, tok + 32 * kWaves, last16, lane);

        // scores, transposed: lane (m, g) gets tokens 16h + 4g + i of row m
        f32x4_t s[RT][2];
        bool kbad = T.lost[0] || T.lost[1];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int x = 0; x < Tile<D>::KS; ++x) kbad = kbad || T.ks[h][x] > kTopScale;
        const bool any_kbad = __builtin_amdgcn_ballot_w64(kbad) != 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          Frag kf[D / 32];
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            const float scale = __uint_as_float(T.ks[h][D == 256 ? c >> 2 : 0] << 23);
#pragma unroll
            for (int p = 0; p < 4; ++p) kf[c].w[p] = widen_byte(T.k[h][c], scale, p);
          }
          if (any_kbad) {   // a NaN block, or a page that does not exist
#pragma unroll
            for (int c = 0; c < D / 32; ++c)
#pragma unroll
              for (int p = 0; p < 4; ++p)
                kf[c].w[p] = T.lost[h] || T.ks[h][D == 256 ? c >> 2 : 0] > kTopScale ? 0x7FC07FC0u : kf[c].w[p];
          }
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            s[rt][h] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int c = 0; c < D / 32; ++c)
              s[rt][h] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf[c].get(), q[rt][c].get(), s[rt][h], 0, 0, 0);
          }
        }
        const bool edge = tok < lo_all || tok + 32 > hi_all;
        const int rel = (int)(tok - first) + 4 * g;
        Frag pf[RT];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          float f[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) f[j] = s[rt][j >> 2][j & 3];
          if (edge) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int t = rel + 16 * (j >> 2) + (j & 3);
              f[j] = t >= row_lo[rt] && t < row_hi[rt] ? f[j] : -__builtin_inff();
            }
          }
          float top = __builtin_fmaxf(__builtin_fmaxf(__builtin_fmaxf(f[0], f[1]), __builtin_fmaxf(f[2], f[3])),
                                      __builtin_fmaxf(__builtin_fmaxf(f[4], f[5]), __builtin_fmaxf(f[6], f[7])));
          top = row_max(top) * a.scale_log2;
          if (__builtin_amdgcn_ballot_w64(top > run_m[rt]) != 0) {
            const float nm = __builtin_fmaxf(run_m[rt], top);
            // nothing seen yet: both are -inf, and there is nothing to rescale
            const float alpha = run_m[rt] == -__builtin_inff() ? 0.0f : __builtin_amdgcn_exp2f(run_m[rt] - nm);
            run_m[rt] = nm;
            run_l[rt] *= alpha;
#pragma unroll
            for (int cb = 0; cb < CB; ++cb) acc[rt][cb] *= alpha;
          }
          const float off = run_m[rt] == -__builtin_inff() ? 0.0f : run_m[rt];
          float sum = 0.0f;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            f[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(f[j], a.scale_log2, -off));
            sum += f[j];
          }
          run_l[rt] += sum;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const f32x2_t two = {f[2 * j], f[2 * j + 1]};
            pf[rt].w[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(two, bf16x2_t));
          }
        }

        // V scales of the lane's eight tokens
        float sc[2][4];
        bool vbad = false;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int q8 = D == 64 ? m >> 3 : D == 128 ? m >> 2 : (m >> 1) & 3;
            uint32_t byte = (T.vs[h][j] >> (8 * q8)) & 0xFFu;
            // behind the end of the sequence lies whatever the page held
            if (edge && tok + 16 * h + 4 * g + j >= len) byte = 0;
            vbad = vbad || byte > kTopScale;
            sc[h][j] = __uint_as_float(byte << 23);
          }
        if (__builtin_amdgcn_ballot_w64(vbad) != 0) {
          // NaN blocks among the values. A masked probability is 0 and 0 * NaN
          // would reach rows that do not see the token, so such blocks enter
          // the product as zeros, and NaN goes to the rows that see them.
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const bool bad = sc[h][j] > __uint_as_float(kTopScale << 23) || sc[h][j] != sc[h][j];
#pragma unroll
              for (int x = 0; x < Tile<D>::VW; ++x) T.v[h][j][x] = bad ? 0u : T.v[h][j][x];
              const uint64_t who = __builtin_amdgcn_ballot_w64(bad);
              sc[h][j] = bad ? 1.0f : sc[h][j];
              if (who == 0) continue;
              // lane 16 G + M reports token 16h + 4G + j, channels M * D/16 and on
              for (int G = 0; G < 4; ++G) {
                const int t = (int)(tok - first) + 16 * h + 4 * G + j;
#pragma unroll
                for (int rt = 0; rt < RT; ++rt) {
                  const bool sees = t >= row_lo[rt] && t < row_hi[rt];
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    const bool hit = sees && (who >> (16 * G + 4 * g + i) & 1);
#pragma unroll
                    for (int cb = 0; cb < CB; ++cb) acc[rt][cb][i] = hit ? __builtin_nanf("") : acc[rt][cb][i];
                  }
                }
              }
            }
        }

        // out += V^T P^T: two 16-channel blocks per byte of codes
#pragma unroll
        for (int p = 0; p < CB / 2; ++p) {
          Frag even, odd;
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int j = 0; j < 4; j += 2) {
              const uint32_t x = widen_byte(T.v[h][j][p >> 2], sc[h][j], p & 3);
              const uint32_t y = widen_byte(T.v[h][j + 1][p >> 2], sc[h][j + 1], p & 3);
              even.w[2 * h + j / 2] = __builtin_amdgcn_perm(y, x, 0x05040100u);
              odd.w[2 * h + j / 2] = __builtin_amdgcn_perm(y, x, 0x07060302u);
            }
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            acc[rt][2 * p] =
                __builtin_amdgcn_mfma_f32_16x16x32_bf16(even.get(), pf[rt].get(), acc[rt][2 * p], 0, 0, 0);
            acc[rt][2 * p + 1] =
                __builtin_amdgcn_mfma_f32_16x16x32_bf16(odd.get(), pf[rt].get(), acc[rt][2 * p + 1], 0, 0, 0);
          }
        }
      }
    }

    // Join the four waves: one row tile at a time through LDS.
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      run_l[rt] = swap_add32(swap_add16(run_l[rt]));
      __syncthreads();   // the buffer's last readers are done
      if (g == 0) {
        red_m[wave * 16 + m] = run_m[rt];
        red_l[wave * 16 + m] = run_l[rt];
      }
      // lane (m, g) holds row m, channels (4g + i) * D/16 + cb
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int cb = 0; cb < CB; cb += 4) {
          const f32x4_t v = {acc[rt][cb][i], acc[rt][cb + 1][i], acc[rt][cb + 2][i], acc[rt][cb + 3][i]};
          *reinterpret_cast<f32x4_t*>(&red[(wave * 16 + m) * LD + (4 * g + i) * CB + cb]) = v;
        }
      __syncthreads();
      const int row = threadIdx.x >> 4;                 // 16 threads per row
      const int col = (threadIdx.x & 15) * (D / 16);    // D/16 channels each
      const int64_t r = r0 + rt * 16 + row;
      float top = -__builtin_inff();
      float w[kWaves], l = 0.0f;
#pragma unroll
      for (int x = 0; x < kWaves; ++x) top = __builtin_fmaxf(top, red_m[x * 16 + row]);
#pragma unroll
      for (int x = 0; x < kWaves; ++x) {
        const float mx = red_m[x * 16 + row];
        // a wave that saw only NaN scores has no maximum, but a NaN sum to pass on
        w[x] = mx == -__builtin_inff() ? (red_l[x * 16 + row] == 0.0f ? 0.0f : 1.0f) : __builtin_amdgcn_exp2f(mx - top);
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
        const int64_t i = r / a.group;
        const int head = hk * a.group + (int)(r - i * a.group);
        if (joined) {
          const int64_t at = ((q0 + i) * heads_q + head) * a.splits + split;
#pragma unroll
          for (int e = 0; e < D / 16; e += 4)
            *reinterpret_cast<f32x4_t*>(a.part_o + at * D + col + e) = f32x4_t{o[e], o[e + 1], o[e + 2], o[e + 3]};
          if ((threadIdx.x & 15) == 0) {
            a.part_ml[at * 2] = top;
            a.part_ml[at * 2 + 1] = l;
          }
        } else {
          const bool empty = hi_of(i) <= lo_of(i);      // a row that sees nothing is zero
          const float inv = empty ? 0.0f : 1.0f / l;
          char* p = static_cast<char*>(a.out) + ((q0 + i) * a.ldo + (int64_t)head * D + col) * 2;
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
    __syncthreads();
  }
}

// Joins the chunks of rows whose cache was split: a wave per (query, head),
// D/64 channels per lane. The row's chunk count follows from the same
// arithmetic as in qknorm_attend; rows written there already are left alone.
template <int D>
__global__ void __launch_bounds__(256) qknorm_attend_join(const AttendArgs a, int row_tile, int64_t max_q) {
  constexpr int E = D / 64;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int heads_q = a.heads_k * a.group;
  const int64_t per_seq = max_q * heads_q;
  const int64_t unit = (int64_t)blockIdx.x * 4 + wave;
  const int64_t b = unit / per_seq;
  if (b >= a.B) return;
  int64_t q0 = b, nq = 1;
  if (a.cu_q) {
    q0 = a.cu_q[b];
    int64_t q1 = a.cu_q[b + 1];
    q0 = q0 < 0 ? 0 : q0 > a.T ? a.T : q0;
    q1 = q1 < q0 ? q0 : q1 > a.T ? a.T : q1;
    nq = q1 - q0;
  }
  int64_t len = a.seq_lens[b];
  len = len < 0 ? 0 : len > a.table_tokens ? a.table_tokens : len;
  const int64_t u0 = unit - b * per_seq;
  const int head = (int)(u0 % heads_q);
  for (int64_t i = u0 / heads_q; i < nq; i += max_q) {
    const int64_t rows = nq * a.group;
    const int64_t r0 = (i * a.group + head % a.group) / (16 * row_tile) * (16 * row_tile);
    const int64_t r_end = rows < r0 + 16 * row_tile ? rows : r0 + 16 * row_tile;
    const int64_t i_first = r0 / a.group, i_last = (r_end - 1) / a.group;
    const int64_t base = len - nq;
    const int64_t pos = base + i_last;
    const int64_t hi = pos < 0 ? 0 : a.causal ? pos + 1 : len;
    const int64_t wlo = base + i_first - a.window + 1;
    const int64_t lo = a.window && wlo > 0 ? wlo : 0;
    const int64_t chunks = hi > lo ? (hi - (lo & ~(int64_t)31) + a.chunk - 1) / a.chunk : 0;
    if (chunks <= 1) continue;
    const int n = (int)(chunks < a.splits ? chunks : a.splits);
    const int64_t at = ((q0 + i) * heads_q + head) * a.splits;
    const float* ml = a.part_ml + at * 2;
    float top = -__builtin_inff();
    for (int s = lane; s < n; s += 64) top = __builtin_fmaxf(top, ml[2 * s]);
    for (int x = 1; x < 64; x <<= 1) top = __builtin_fmaxf(top, __shfl_xor(top, x));
    float l = 0.0f, o[E];
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] = 0.0f;
    const float* po = a.part_o + at * D + lane * E;
#pragma unroll 4
    for (int s = 0; s < n; ++s) {
      const float ms = ml[2 * s], ls = ml[2 * s + 1];
      const float w = ms == -__builtin_inff() ? (ls == 0.0f ? 0.0f : 1.0f) : __builtin_amdgcn_exp2f(ms - top);
      l += w * ls;
#pragma unroll
      for (int e = 0; e < E; ++e) o[e] += w * po[(int64_t)s * D + e];
    }
    const int64_t my_pos = base + i;
    const int64_t my_hi = my_pos < 0 ? 0 : a.causal ? my_pos + 1 : len;
    const int64_t my_lo0 = my_pos - a.window + 1;
    const int64_t my_lo = a.window && my_lo0 > 0 ? my_lo0 : 0;
    const bool empty = my_hi <= my_lo;
    const float inv = 1.0f / l;
    __bf16* p = static_cast<__bf16*>(a.out) + (q0 + i) * a.ldo + (int64_t)head * D + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) p[e] = (__bf16)(empty ? 0.0f : o[e] * inv);
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
    int64_t mq = p.max_q;
    void* jargs[] = {&a, &rt, &mq};
    const int64_t units = (int64_t)a.B * mq * a.heads_k * a.group;
    const void* join = p.head_dim == 64    ? reinterpret_cast<const void*>(qknorm_attend_join<64>)
                       : p.head_dim == 128 ? reinterpret_cast<const void*>(qknorm_attend_join<128>)
                                           : reinterpret_cast<const void*>(qknorm_attend_join<256>);
    e = hipLaunchKernel(join, dim3((unsigned)((units + 3) / 4)), dim3(256), jargs, 0,
                        static_cast<hipStream_t>(stream));
  }
  if (e != hipSuccess) {
    *err = std::string("kernel launch: ") + hipGetErrorString(e);
    return (int)e;
  }
  return 0;
}

}  // namespace qkn

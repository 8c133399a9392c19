// Reading a paged key / value cache back as rows, on gfx950 (CDNA4): token t's
// keys and values, from the slot it names, as elements of the row type. Codes are
// widened with their scale applied, exactly (a code has at most four significant
// bits; bf16 holds those of values below 2^-130 only in part).
//
// It streams: bound by HBM. A lane takes 16 bytes of the rows written (one element
// where they are not aligned), and a wave 64 of them of one token's K or V, so that
// the slot and the side are scalar, for four tokens, whose loads are in flight
// together (8 heads of 128, 16384 tokens of MXFP8 into bf16: 18.0 us, 5.7 TB/s, 20.2
// with one token a wave; into float32 with 32 bytes a lane in two stores 45 us,
// now 26.6; MXFP4 15.5, rows 25.2).

#include "qknorm_rope_device.hpp"

#include <string>
#include <type_traits>

namespace qkn {
namespace {

constexpr int kGatherTokens = 4;

// PB: bytes of a piece where rows are copied; for codes, 16 where the rows written
// take 16-byte stores.
template <class IO, int KIND, int PB>
__global__ void __launch_bounds__(64 * kRopeWaves) qknorm_gather(const GatherArgs a) {
  const int lane = threadIdx.x & 63;
  const uint32_t unit = blockIdx.x * kRopeWaves + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (unit >= a.units) return;
  const uint32_t t0 = over(unit, a.by_groups);
  const int group = unit - t0 * a.by_groups.d;
  const int per_side = a.out[0] && a.out[1] ? a.groups >> 1 : a.groups;
  const int side = a.out[0] ? (group >= per_side ? 1 : 0) : 1;
  const int item = (side && a.out[0] ? group - per_side : group) * 64 + lane;
  const bool on = item < a.items;
  const int head = on ? over(item, a.by_pieces) : 0, piece = on ? item - head * a.pieces : 0;   // idle lanes: the first

  // A piece as it is loaded: rows, or codes and their scale byte.
  constexpr bool CODES = KIND != GATHER_ROWS;
  constexpr int VW = IO::kVW;                               // elements of codes
  using MX = std::conditional_t<KIND == GATHER_MXFP8, Mx8, Mx4>;
  struct In {
    Piece<CODES ? 16 : PB> x;
    Codes<MX, VW> q;
    int byte;
    bool live;
  };
  const auto load = [&](In& in, int64_t t) {
    const int64_t slot = load_uniform(a.slots + t);
    in.live = slot >= 0 && slot < a.n_tokens_held;          // a row that holds no token: slot 0, not stored
    const int64_t at = in.live ? slot : 0;
    const int64_t page = at >> a.log2_page, off = at & (((int64_t)1 << a.log2_page) - 1);
    const char* p = a.cache[side] + page * a.page_stride + off * a.token_stride + head * a.head_stride;
    if constexpr (CODES) {
      load_bytes<VW * MX::kBits / 8, false>(p + piece * (VW * MX::kBits / 8), in.q.w);
      in.byte = a.scales[side][page * a.scale_page_stride + off * (a.head_dim >> 5) + head * a.scale_head_stride + piece / (32 / VW)];
    } else {
      load_bytes<PB, true>(p + piece * PB, in.x.w);
    }
  };
  const auto store = [&](const In& in, int64_t t) {
    if (!in.live || !on) return;
    char* y = a.out[side] + t * a.ld[side];
    if constexpr (!CODES) {
      store_bytes<PB>(y + ((int64_t)head * a.pieces + piece) * PB, in.x.w);
    } else {
      float f[VW];
      code_values<MX, VW>(in.q, in.byte > MX::kTop ? 0xFF : in.byte, f);
      uint32_t o[4];
      narrow<IO, VW>(f, o);
      y += ((int64_t)head * a.head_dim + piece * VW) * IO::kBytes;
      if constexpr (PB == 16) {
        store_bytes<16>(y, o);
      } else {
#pragma unroll
        for (int e = 0; e < VW; ++e) {
          const uint32_t one = IO::kBytes == 4 ? o[e] : o[e >> 1] >> (16 * (e & 1));
          store_bytes<IO::kBytes>(y + e * IO::kBytes, &one);
        }
      }
    }
  };
  // kGatherTokens tokens at a time, so that their loads are in flight together
  for (int64_t t = t0 * (int64_t)kGatherTokens; t < a.T; t += a.tokens * kGatherTokens) {
    In in[kGatherTokens];
#pragma unroll
    for (int k = 0; k < kGatherTokens; ++k) load(in[k], t + k < a.T ? t + k : t);
#pragma unroll
    for (int k = 0; k < kGatherTokens; ++k)
      if (t + k < a.T) store(in[k], t + k);
  }
}

using GatherFn = void (*)(const GatherArgs);

template <class IO>
GatherFn pick_gather(int kind, bool wide) {
  switch (kind) {
    case GATHER_ROWS:
      return wide ? qknorm_gather<IO, GATHER_ROWS, 16> : qknorm_gather<IO, GATHER_ROWS, IO::kBytes>;
    case GATHER_MXFP4:
      return wide ? qknorm_gather<IO, GATHER_MXFP4, 16> : qknorm_gather<IO, GATHER_MXFP4, IO::kBytes>;
    default:
      return wide ? qknorm_gather<IO, GATHER_MXFP8, 16> : qknorm_gather<IO, GATHER_MXFP8, IO::kBytes>;
  }
}

}  // namespace

int launch_gather(int kind, int dtype, int piece_bytes, const GatherArgs& args, void* stream, std::string* err) {
  GatherArgs a = args;
  const GatherFn fn = dtype == kDtypeBF16 ? pick_gather<BF16>(kind, piece_bytes == 16) : pick_gather<F32>(kind, piece_bytes == 16);
  // waves of the first a.tokens runs of kGatherTokens tokens; the rest loop (a
  // launch holds fewer than 2^32 threads)
  constexpr int64_t kMostBlocks = (int64_t)1 << 22;
  const int64_t most = (grid_cap() < kMostBlocks ? grid_cap() : kMostBlocks) * kRopeWaves / a.groups;
  const int64_t runs = (a.T + kGatherTokens - 1) / kGatherTokens;
  a.tokens = runs < most ? runs : most > 0 ? most : 1;
  a.units = (uint32_t)(a.tokens * a.groups);
  a.by_groups = divisor((uint32_t)a.groups);
  a.by_pieces = divisor((uint32_t)a.pieces);
  void* kargs[] = {&a};
  const hipError_t e = hipLaunchKernel(reinterpret_cast<const void*>(fn), dim3((a.units + kRopeWaves - 1) / kRopeWaves),
                                       dim3(64 * kRopeWaves), kargs, 0, static_cast<hipStream_t>(stream));
  if (e == hipSuccess) return 0;
  *err = std::string("kernel launch: ") + hipGetErrorString(e);
  return (int)e;
}

}  // namespace qkn

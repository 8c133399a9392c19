// Reading a paged key / value cache back as rows, on gfx950 (CDNA4): token t's
// keys and values, from the slot it names, as elements of the row type. Codes are
// widened with their scale applied, exactly (a code has at most four significant
// bits).
//
// It streams: bound by HBM. A lane takes one piece of a head, eight elements of a
// quantised cache (16 bytes as bf16) or 16 bytes of rows; a wave takes 64 pieces of
// one token's K or V, so that the slot and the side are scalar.

#include "qknorm_rope_device.hpp"

#include <string>
#include <type_traits>

namespace qkn {
namespace {

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
  const int head = over(item, a.by_pieces), piece = item - head * a.pieces;
  const bool on = item < a.items;

  for (int64_t t = t0; t < a.T; t += a.tokens) {
    const int64_t slot = load_uniform(a.slots + t);
    if (slot < 0 || slot >= a.n_tokens_held) continue;      // a row that holds no token
    if (!on) continue;
    const int64_t page = slot >> a.log2_page, off = slot & (((int64_t)1 << a.log2_page) - 1);
    const char* p = a.cache[side] + page * a.page_stride + off * a.token_stride + head * a.head_stride;
    char* y = a.out[side] + t * a.ld[side];
    if constexpr (KIND == GATHER_ROWS) {
      Piece<PB> x;
      load_bytes<PB, true>(p + piece * PB, x.w);
      store_bytes<PB>(y + ((int64_t)head * a.pieces + piece) * PB, x.w);
    } else {
      using MX = std::conditional_t<KIND == GATHER_MXFP8, Mx8, Mx4>;
      Codes<MX, 8> q;
      load_bytes<MX::kBits, false>(p + piece * MX::kBits, q.w);
      int byte = a.scales[side][page * a.scale_page_stride + off * (a.head_dim >> 5) + head * a.scale_head_stride + (piece >> 2)];
      if (byte > MX::kTop) byte = 0xFF;
      float f[8];
      code_values<MX, 8>(q, byte, f);
      uint32_t o[IO::kBytes * 2];
      narrow<IO, 8>(f, o);
      y += ((int64_t)head * a.head_dim + piece * 8) * IO::kBytes;
      if constexpr (PB == 16) {
#pragma unroll
        for (int q4 = 0; q4 < IO::kBytes / 2; ++q4) store_bytes<16>(y + 16 * q4, o + 4 * q4);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t one = IO::kBytes == 4 ? o[e] : o[e >> 1] >> (16 * (e & 1));
          store_bytes<IO::kBytes>(y + e * IO::kBytes, &one);
        }
      }
    }
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
  // waves of the first a.tokens tokens; the rest of the tokens loop (a launch
  // holds fewer than 2^32 threads)
  constexpr int64_t kMostBlocks = (int64_t)1 << 22;
  const int64_t most = (grid_cap() < kMostBlocks ? grid_cap() : kMostBlocks) * kRopeWaves / a.groups;
  a.tokens = a.T < most ? a.T : most > 0 ? most : 1;
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

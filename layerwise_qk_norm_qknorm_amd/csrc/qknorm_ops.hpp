// Internal interface between the C ABI layer of the operators around headwise
// QK-Norm (qknorm_ops_api.cpp: validation and planning, no HIP calls) and
// their kernels (qknorm_rope.hip, qknorm_rope_paired.hip, qknorm_attend.hip,
// qknorm_attend_wide.hip, qknorm_gather.hip).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <string>

namespace qkn {

// Unsigned division by a constant of the launch, for numerators below 2^31:
// n / d = n * mul >> (31 + shift) with mul = ceil(2^(31 + shift) / d) and
// shift = ceil(log2 d) (Granlund and Montgomery's round-up method).
struct Divisor {
  uint32_t mul = 0, shift = 0, d = 1;
};
inline Divisor divisor(uint32_t d) {
  Divisor r;
  r.d = d;
  while (((uint64_t)1 << r.shift) < d) ++r.shift;
  r.mul = (uint32_t)((((uint64_t)1 << (31 + r.shift)) + d - 1) / d);
  return r;
}

// Widest head of the rotation kernels (columns).
constexpr int kRopeMaxHead = 1024;

// How the rotation kernels spread a head over lanes. A lane holds pieces in
// pairs (A, B): the two sides of the half-split rotation, so that no lane
// needs another's elements to rotate its own. `vw` elements make a piece
// (16 or 8 bytes of the row type, or one element); pair p of a head is held
// by lane p mod `lanes` of the head's group.
struct RopePlan {
  int whole = 0;        // 1: one 16-byte chunk of a head per lane (qknorm_rope.hip); the fields up to
                        // `pairs` describe the other layout (qknorm_rope_paired.hip)
  int piece_bytes = 0;  // 16, 8 or the element size
  int vw = 1;           // elements per piece
  int pairs = 0;        // pairs per head
  int lanes = 0;        // lanes per head: a power of two, 1..64
  int np = 1;           // pairs per lane: 1, or up to 8 on the element path
  int slots = 1;        // wave passes (64 / lanes heads each) per wave
  int waves = 1;        // waves per token in one block
  int tokens = 1;       // tokens per block
  int groups = 1;       // one chunk per lane: waves per token
  int apart = 0;        // 1 (MXFP4): a launch for Q and one for K and V
};

// Positions on several axes (time, height, width): the axis of every angle, two
// bits each, and how far apart the axes' positions lie.
constexpr int kMostAxes = 4;
struct RopeAxes {
  int n;               // 0: one position a token
  int64_t ld;
  uint32_t of[kRopeMaxHead / 2 / 16];
};

struct RopeSide {  // one of Q, K, V
  const void* x;
  void* y;
  const void* gamma;   // NULL: not normalized
  int64_t ldx, ldy;
  int heads;
};

struct RopeArgs {
  RopeSide side[3];
  int first[3];        // slot (one chunk per lane: wave) where each side begins; neither mixes sides
  int n_slots;         // slots of a token
  int64_t T;
  int64_t gstride;
  int head_dim;
  int pairs, rot_pairs, rot;
  int log2_lanes;
  int half_lanes;      // one chunk per lane, half-split: lanes between the members of a pair
  int idle;            // 1: a head leaves some lanes or a side of a pair empty
  int waves, tokens;   // of a block: waves per token, tokens
  uint32_t waves_inv;  // 65536 / waves, rounded up
  // one chunk per lane: waves per token, waves of the launch; `tokens` is then the tokens these cover
  Divisor by_groups;
  uint32_t units;
  const float* cos_sin;
  int64_t ld_table, n_positions;
  const int64_t* positions;
  float inv_div, eps;
  // appending only
  const int64_t* slots;
  int64_t n_tokens_held;   // n_pages * page_size
  int log2_page;
  char* cache[2];          // K, V
  char* scales[2];
  int64_t page_stride, head_stride, token_stride;   // bytes
  int64_t scale_page_stride, scale_head_stride;     // bytes
  int y_wide;              // 1: the rows for cached values take 16-byte stores
};

struct RopeAxesArgs : RopeArgs {   // of the kernels for several axes; the others take what it begins with
  RopeAxes axes;
};

constexpr int kRopeMaxWaves = 8;   // of a block, paired layout
constexpr int kRopeWaves = 4;      // of a block, one chunk per lane

enum RopeMode : int { ROPE_FORWARD = 0, ROPE_APPEND_ROWS = 1, ROPE_APPEND_MXFP4 = 2, ROPE_APPEND_MXFP8 = 3 };

int launch_rope(int mode, int dtype, bool interleaved, const RopePlan& plan, const RopeAxesArgs& args, void* stream,
                std::string* err);

struct RopeGradSide {
  const void* x;
  const void* dy;
  void* dx;
  const void* gamma;
  float* dgamma;       // NULL: not wanted
  int64_t ldx, lddy, lddx;
  int heads;
};

struct RopeGradArgs {
  RopeGradSide side[2];
  int first[2];
  int n_slots;
  int64_t T;
  int64_t gstride;
  int head_dim;
  int pairs, rot_pairs, rot;
  int log2_lanes;
  int half_lanes;
  int idle;
  int workers;         // token workers (blocks) per slot
  const float* cos_sin;
  int64_t ld_table, n_positions;
  const int64_t* positions;
  float inv_div, eps;
  float* partial;      // [rows][head_dim], see rope_grad_rows
};
struct RopeGradAxesArgs : RopeGradArgs {
  RopeAxes axes;
};

constexpr int kGradWaves = 4;   // waves of a gradient block, each with tokens of its own

// The kernel of the paired layout for a plan (NULL: none).
const void* rope_paired_kernel(int mode, int dtype, bool interleaved, bool axes, const RopePlan& plan);
const void* rope_paired_grad_kernel(int dtype, bool interleaved, bool axes, const RopePlan& plan);

// Rows of partial gamma gradients a launch writes.
int64_t rope_grad_rows(const RopeGradArgs& a);

int launch_rope_grad(int dtype, bool interleaved, const RopePlan& plan, const RopeGradAxesArgs& args, void* stream,
                     std::string* err);

struct AttendArgs {
  const void* q;         // [T][heads_q * head_dim] bf16
  void* out;
  int64_t ldq, ldo;
  int T;
  const uint8_t* cache[2];    // K, V codes
  const uint8_t* scales[2];
  int64_t page_stride, head_stride, scale_page_stride, scale_head_stride;   // bytes
  int64_t token_stride;       // bytes
  int scale_row;              // scale bytes of a token's head
  uint32_t n_pages;      // at most 2^31 - 1: ids are int32
  int log2_page;
  int heads_k, group;    // query heads per key head
  const int32_t* table;
  int64_t ld_table;
  int table_tokens;      // tokens a table row can name
  const int32_t* seq_lens;
  const int32_t* cu_q;   // NULL: one query per sequence
  int B;
  int causal;
  int window;            // 0: none
  float scale_log2;      // scale * log2(e)
  Divisor by_group, by_pairs, by_splits, by_heads;   // pairs: B * heads_k
  int row_tiles;         // blocks along a sequence's rows (each loops over the rest)
  int splits;            // blocks along the cache
  int chunk;             // cached tokens a block takes at a time, a multiple of 128
  float* part_o;         // [T][heads_q][splits][head_dim]
  float* part_ml;        // [T][heads_q][splits][2]: maximum (base 2), sum
};

struct AttendPlan {
  int head_dim = 0;
  int row_tile = 1;      // 16-row tiles per block: 1, 2 or 4; wide caches 1, 2, 8 or 16
  int row_tiles = 1;
  int splits = 1;
  int most_splits = 1;   // what the workspace is sized for: no smaller for a longer max_len
  int chunk = 0;
  int64_t max_q = 1;
};

int launch_attend(const AttendPlan& plan, const AttendArgs& args, void* stream, std::string* err);

// Adds up the parts of rows whose cache was split.
int launch_attend_join(const AttendPlan& plan, const AttendArgs& args, void* stream, std::string* err);

// Caches of bf16 rows and MXFP8 (mx8). row_tile 1 and 2: the kernel whose waves
// share a block's rows; 8 and 16: the one whose four or eight waves take 32 each.
int launch_attend_wide(bool mx8, const AttendPlan& plan, const AttendArgs& args, void* stream, std::string* err);

struct GatherArgs {
  const char* cache[2];    // K, V; NULL out: not wanted
  const uint8_t* scales[2];
  char* out[2];
  int64_t ld[2];           // bytes
  int64_t page_stride, head_stride, token_stride, scale_page_stride, scale_head_stride;   // bytes
  const int64_t* slots;
  int64_t T, n_tokens_held;
  int log2_page;
  int head_dim;
  int pieces;              // of a token's head
  int items;               // pieces of a token's heads
  int groups;              // waves of 64 items that a token's heads take
  Divisor by_pieces, by_groups;
  uint32_t units;          // waves of the launch
  int64_t tokens;          // runs of tokens that these cover; the rest loop
};
enum GatherKind : int { GATHER_ROWS = 0, GATHER_MXFP4 = 1, GATHER_MXFP8 = 2 };
// piece_bytes: of the rows' loads and stores, 16 or one element (codes: of the stores; a piece is 16 bytes of rows).
int launch_gather(int kind, int dtype, int piece_bytes, const GatherArgs& args, void* stream, std::string* err);

}  // namespace qkn

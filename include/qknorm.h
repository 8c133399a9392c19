/*
 * qknorm.h -- layerwise QK-Norm on one MI355X (gfx950), as a C ABI.
 *
 * Library: libqknorm.so (HIP kernels for gfx950 behind plain C entry points).
 *
 * What is computed
 * ----------------
 * Source: "SwiftQK: Fast and Communication-Efficient Tensor Parallelism for
 * Query-Key Normalization" (Kim, Han, Kim; arXiv 2608.09160v1).
 *
 * Layerwise QK-Norm (introduction of the paper) normalizes each token's whole
 * projected Q vector with one RMS factor and, independently, its whole
 * projected K vector with another, before attention; V is not touched. For one
 * vector x of full width H, RMS-Norm (Eq. 1; its body is missing from the
 * page text, and this library reads it as the standard RMSNorm) is
 *
 *     y_j = x_j * gamma_j / sqrt( (sum_i x_i^2) / H + eps ).
 *
 * Phase A of the paper: the only cross-shard quantity the factor needs is the
 * plain sum of squares, so each column shard of x produces one float32
 * partial sum and the global sum is the float32 sum of the partials. Phase B
 * and the final scaling: each element is multiplied by gamma_j (independent
 * of the global sum) and then by the factor r = 1/sqrt(sum/H + eps).
 *
 * Arithmetic (identical in every entry point, so results compose bit for bit):
 *   - inputs are widened exactly to float32;
 *   - partial[s] = float32 sum of x_j^2 over shard s, in a fixed order that
 *     depends only on the shapes, the shard count and T;
 *   - sum = ((partial[0] + partial[1]) + ...) + partial[S-1]   (float32);
 *   - m = fma(sum, 1/H, eps), with 1/H rounded once to float32 on the host;
 *   - r = reciprocal square root of m from the hardware's float32 rsqrt
 *     (within about one float32 ulp; where m would fall below the float32
 *     normal range it is formed from 2^64 * sum and 2^64 * eps instead, both
 *     exact, and r is scaled back by 2^32, keeping that accuracy);
 *   - y_j = (x_j * gamma_j) * r, rounded once to the I/O type (bf16 and FP8:
 *     round to nearest even; FP8 saturates to +-448).
 *   The float32 accumulation is the paper's (Fig. 2(b) accumulates squared
 *   sums in FP32 for BF16 activations); rows whose sum of squares overflows
 *   float32 (|x| around 1e19) give 0 or NaN instead of the real result, and
 *   rows whose squares fall below the float32 normal range (|x| below about
 *   1e-19) lose accuracy in the sum (with eps = 0 and |x| below about 1e-23
 *   the squares vanish and the result is inf or NaN).
 *
 * Data layout
 * -----------
 * An operand describes one of Q or K as row-major rows in device memory:
 * element (t, j) of the input is x[t * ld_x + j], 0 <= t < T, 0 <= j < h.
 * A packed QKV buffer [T, Hq + Hk + Hv] is described by two operands with
 * the same ld (Hq + Hk + Hv): Q at column 0, K at column Hq. V columns and
 * any other memory are never read or written.
 *
 * A shard count S splits each of Q and K into S contiguous column shards of
 * width h/S (h % S == 0 is required): shard s covers columns [s*h/S,
 * (s+1)*h/S). This emulates one rank's view under tensor parallelism.
 *
 * Ownership and streams
 * ---------------------
 * The caller owns every buffer. The library allocates nothing and keeps no
 * state except a per-thread error message. Work is enqueued on `stream` (a
 * hipStream_t; NULL means the default stream of the calling thread's current
 * device) and the call returns without synchronizing. The kernel runs on the
 * stream's device; all pointers are device pointers that this device can
 * access. Calls on different streams or threads are independent; two calls
 * whose outputs overlap race, as any two kernels would. The kernels are
 * built for gfx950 only. The environment variable QKNORM_MAX_GRID, read once
 * when the library first launches a kernel, caps the number of blocks per
 * launch (blocks then loop over several token groups), which leaves compute
 * units to kernels running beside these on other streams; results do not
 * depend on it. qknorm_headwise_rope, qknorm_paged_append (with several axes too)
 * and qknorm_paged_gather launch at least the blocks that one token's heads take;
 * the gradients and the attention size their grids themselves.
 *
 * Errors
 * ------
 * Argument errors return QKNORM_ERR_INVALID_ARG before anything is launched
 * and nothing is written; QKNORM_ERR_UNSUPPORTED means valid arguments that
 * this library cannot run (a row wider than the kernels hold). With one
 * shard a token's Q plus K columns may span up to 8192 16-byte chunks for
 * bf16 and fp32 and 4096 for FP8 (65536 bf16 / 32768 fp32 / 65536 FP8
 * elements) on the 16-byte path, and about 4096 / 6144 / 2048 chunks on the
 * element-wise path. With S > 1 shards each shard takes a power-of-two lane
 * group of at most 1024/S lanes, so a shard holds proportionally fewer.
 * QKNORM_ERR_HIP means a HIP runtime call failed. qknorm_last_error() gives
 * the message.
 * Faults inside kernels surface at the caller's next synchronization. T == 0
 * is a no-op that returns QKNORM_OK after the scalar arguments are checked.
 * Pointers must be aligned to their element size (bf16 and bf16 gamma: 2
 * bytes; fp32, fp32 gamma and the float32 statistics: 4 bytes); a
 * misaligned element pointer is an argument error. Pointers or strides that
 * are not 16-byte multiples, or shard widths that are not a multiple of 16
 * bytes of elements, are not errors: they run a slower element-wise path
 * with bit-identical results.
 */
#ifndef QKNORM_H
#define QKNORM_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define QKNORM_ABI_VERSION 3

/* Largest shard count and number of statistic planes accepted. */
#define QKNORM_MAX_SHARDS 64
#define QKNORM_MAX_PLANES 64
/* Largest full width H accepted by qknorm_apply_with_stats (exact in float32). */
#define QKNORM_MAX_FULL_WIDTH (1 << 24)

typedef enum qknorm_dtype {
  QKNORM_F32 = 0,      /* float32 rows and gamma */
  QKNORM_BF16 = 1,     /* bfloat16 rows and gamma, float32 arithmetic */
  QKNORM_FP8_E4M3 = 2  /* FP8 E4M3 rows (OCP E4M3FN: bias 7, max 448, NaN 0x7F/0xFF,
                          no infinity), bfloat16 gamma, float32 arithmetic. Outputs are
                          rounded to nearest even and saturated to +-448; NaN stays NaN.
                          Fig. 2(b) of the paper evaluates FP8-E4M3 activations with
                          FP32 accumulation. */
} qknorm_dtype_t;

typedef enum qknorm_status {
  QKNORM_OK = 0,
  QKNORM_ERR_INVALID_ARG = 1,
  QKNORM_ERR_UNSUPPORTED = 2,
  QKNORM_ERR_HIP = 3
} qknorm_status_t;

/* Which entry point a plan is described for (qknorm_describe_plan). */
typedef enum qknorm_op {
  QKNORM_OP_FUSED = 0,
  QKNORM_OP_PARTIAL_STATS = 1,
  QKNORM_OP_APPLY_WITH_STATS = 2
} qknorm_op_t;

/* One of Q or K. */
typedef struct qknorm_operand {
  const void* x;     /* input rows, element (t, j) at x[t*ld_x + j] (elements of the I/O type) */
  int64_t ld_x;      /* input row stride in elements, >= h */
  void* y;           /* output rows, element (t, j) at y[t*ld_y + j]; y == x with ld_y == ld_x
                        is in place; any other overlap with an input or output is rejected.
                        Not used by qknorm_partial_stats (may be NULL there). */
  int64_t ld_y;      /* output row stride in elements, >= h (ignored by qknorm_partial_stats) */
  const void* gamma; /* h per-column scales: the row type, bf16 for FP8 rows
                        (not used by qknorm_partial_stats) */
  int64_t h;         /* local width: number of columns normalized, > 0 */
} qknorm_operand_t;

/*
 * qknorm_fused -- the whole path in one kernel: Phase A partial sums for S
 * shards, their combination, Phase B (x * gamma) and the final scaling
 * (Eq. 1 with H = h, the local width). Each Q/K element is read once and
 * written once.
 *
 *   q, k    operand descriptors (host pointers to structs holding device pointers)
 *   T       tokens (rows), >= 0
 *   dtype   QKNORM_F32, QKNORM_BF16 (x, y and gamma alike) or QKNORM_FP8_E4M3
 *           (x and y FP8, gamma bf16)
 *   eps     finite, >= 0
 *   shards  S in [1, QKNORM_MAX_SHARDS]; q->h % S == 0 and k->h % S == 0
 *   stream  hipStream_t or NULL
 */
int qknorm_fused(const qknorm_operand_t* q, const qknorm_operand_t* k, int64_t T, int dtype,
                 float eps, int shards, void* stream);

/*
 * qknorm_partial_stats -- Phase A alone: the float32 sum of squares of every
 * shard of every row, which is what each tensor-parallel rank would
 * contribute to the exchange.
 *
 *   partials  device float32 [S][2][T]: partials[(s*2 + c)*T + t] is shard s of
 *             Q (c = 0) or K (c = 1) for token t. Must not overlap the inputs.
 *   other arguments as for qknorm_fused (y, ld_y and gamma are ignored).
 */
int qknorm_partial_stats(const qknorm_operand_t* q, const qknorm_operand_t* k, int64_t T,
                         int dtype, int shards, float* partials, void* stream);

/*
 * qknorm_apply_with_stats -- the combination and Phase B / final scaling for a
 * local slice, given the statistic planes received from all shards: the
 * planes are added in order p = 0 .. n_planes-1 in float32 and Eq. 1 divides
 * by the full width (hq_full for Q, hk_full for K), not the local width.
 *
 *   stats     device float32 [n_planes][2][T], same layout as `partials`
 *             (a qknorm_partial_stats output is a valid input, n_planes = S);
 *             n_planes = 1 passes an already combined sum. Must not overlap
 *             the outputs.
 *   n_planes  in [1, QKNORM_MAX_PLANES]
 *   hq_full, hk_full  full widths H, with h <= H_full <= QKNORM_MAX_FULL_WIDTH
 *   q, k, T, dtype, eps, stream as for qknorm_fused.
 *
 * qknorm_fused with S shards gives bit-identical outputs to
 * qknorm_partial_stats with S shards followed by this call with n_planes = S
 * and H_full = h.
 */
int qknorm_apply_with_stats(const qknorm_operand_t* q, const qknorm_operand_t* k, int64_t T,
                            int dtype, float eps, const float* stats, int n_planes,
                            int64_t hq_full, int64_t hk_full, void* stream);

/*
 * qknorm_headwise -- headwise QK-Norm: the paper's introduction names this
 * granularity as one independent normalization factor per attention head.
 * Every head (head_dim contiguous columns; Q has q->h / head_dim heads and K
 * has k->h / head_dim) is normalized with Eq. 1 on its own, H = head_dim:
 * y_j = (x_j * gamma_j) * rsqrt(sum over the head of x^2 / head_dim + eps),
 * with the same float32 arithmetic as the layerwise calls. There is no
 * combination across heads, so nothing here needs an exchange between
 * tensor-parallel ranks.
 *
 *   head_dim           > 0; q->h and k->h must be multiples of it
 *   gamma_head_stride  gamma element (head, j) is gamma[head * stride + j]:
 *                      0 shares one [head_dim] vector across heads (the usual
 *                      per-head RMSNorm weight), head_dim reads a full [h]
 *                      vector; any stride >= 0 is accepted
 *   q, k, T, dtype, eps, stream as for qknorm_fused (gamma holds
 *   (heads - 1) * stride + head_dim elements).
 *
 * Heads of up to 4096 bf16 / 2048 fp32 / 8192 FP8 elements and up to 256 heads per
 * token (Q and K together) are supported; larger ones return
 * QKNORM_ERR_UNSUPPORTED.
 */
int qknorm_headwise(const qknorm_operand_t* q, const qknorm_operand_t* k, int64_t T, int dtype,
                    float eps, int64_t head_dim, int64_t gamma_head_stride, void* stream);

/* ------------------------------------------------------------------------
 * Headwise QK-Norm with the position rotation, its gradients, appending to a
 * paged cache, reading it back, and attention over it.
 *
 * The rotation (rotary position embedding) turns each pair (a, b) of a head's
 * first rot_dim columns by its position's angle: (a c - b s, b c + a s). The
 * angles' cos and sin come from a table the caller keeps.
 * ------------------------------------------------------------------------ */

/* Widest head of the calls below (attention has its own widths). */
#define QKNORM_MAX_ROPE_HEAD 1024

/* Where the rotation's angles come from. */
typedef struct qknorm_rope {
  const float* cos_sin;      /* device float32 table [n_positions][rot_dim]: row p holds the cos of
                                position p's rot_dim/2 angles, then their sin */
  int64_t ld;                /* row stride in elements, >= rot_dim */
  int64_t n_positions;       /* rows of the table, > 0 */
  const int64_t* positions;  /* device int64 [T]: each token's position. One outside
                                [0, n_positions) makes the token's rotated columns NaN. */
  int64_t rot_dim;           /* even, in [0, head_dim]: columns of each head that are rotated.
                                0: no rotation, the other fields are not used */
  int interleaved;           /* 0: column i pairs with column i + rot_dim/2;
                                1: column 2i pairs with column 2i + 1 */
} qknorm_rope_t;

/*
 * qknorm_headwise_rope -- headwise QK-Norm (as qknorm_headwise), then the
 * rotation of every head, in one pass: each element is read once and written
 * once, rounded once after the rotation.
 *
 *   rope  the rotation (host pointer); NULL is the same as rot_dim = 0
 *   other arguments as for qknorm_headwise. head_dim <= QKNORM_MAX_ROPE_HEAD.
 *
 * Outputs may be in place (y == x with ld_y == ld_x); the table and positions
 * must not overlap the outputs.
 */
int qknorm_headwise_rope(const qknorm_operand_t* q, const qknorm_operand_t* k, int64_t T, int dtype,
                         float eps, int64_t head_dim, int64_t gamma_head_stride,
                         const qknorm_rope_t* rope, void* stream);

/* Most axes of positions. */
#define QKNORM_MAX_AXES 4

/* Positions on several axes (images and video: time, height, width): each angle
 * takes the position of one of them. */
typedef struct qknorm_axes {
  int n_axes;                /* in [1, QKNORM_MAX_AXES] */
  const uint8_t* axis;       /* host memory, [rot_dim / 2]: the axis of every angle, below n_axes. Read during
                                the call only. */
  int64_t ld_positions;      /* rope->positions is [n_axes][T] with this row stride in elements, >= 0 (0: the
                                axes share one row) */
} qknorm_axes_t;

/*
 * qknorm_headwise_rope_axes -- qknorm_headwise_rope with positions on several
 * axes: angle i of token t is that of position rope->positions[axis[i] *
 * ld_positions + t]. A position outside the table makes the columns that its
 * axis turns NaN.
 *
 *   axes  (host pointer); NULL: one axis, as qknorm_headwise_rope. Not used with
 *         rot_dim = 0.
 *   other arguments as for qknorm_headwise_rope.
 */
int qknorm_headwise_rope_axes(const qknorm_operand_t* q, const qknorm_operand_t* k, int64_t T, int dtype, float eps,
                              int64_t head_dim, int64_t gamma_head_stride, const qknorm_rope_t* rope,
                              const qknorm_axes_t* axes, void* stream);

/* One of Q or K of the backward pass. */
typedef struct qknorm_grad_operand {
  const void* x;     /* the forward call's input rows */
  int64_t ld_x;      /* row strides in elements, >= h */
  const void* dy;    /* gradient of the forward call's output, rows of the row type */
  int64_t ld_dy;
  void* dx;          /* out: gradient of x, rows of the row type. dx == dy or dx == x with the same
                        stride is in place; any other overlap with an input or output is rejected. */
  int64_t ld_dx;
  const void* gamma; /* as in the forward call */
  float* dgamma;     /* out: gradient of gamma, float32, laid out as gamma (overwritten, not added to;
                        elements between heads of a stride > head_dim are left alone). NULL: not wanted */
  int64_t h;
} qknorm_grad_operand_t;

/*
 * qknorm_headwise_rope_backward -- gradients of qknorm_headwise_rope (and with
 * rot_dim = 0 of qknorm_headwise): with g the gradient turned back by the
 * rotation, r the head's factor, xr = x r and gg = g gamma,
 *     dx = r (gg - xr mean(gg xr)),   dgamma_j = sum g_j xr_j
 * over all tokens and over the heads that share gamma. Sums are in a fixed
 * order: the same call gives the same bits.
 *
 *   dtype              QKNORM_F32 or QKNORM_BF16
 *   gamma_head_stride  0 (shared) or >= head_dim
 *   workspace          device memory of at least
 *                      qknorm_headwise_rope_backward_workspace(...) bytes, 16-byte
 *                      aligned, not shared with a call that may run at the same
 *                      time; its contents need no preparation. May be NULL where
 *                      that size is 0.
 * T == 0 launches nothing, and dgamma is then not written.
 */
int qknorm_headwise_rope_backward(const qknorm_grad_operand_t* q, const qknorm_grad_operand_t* k, int64_t T,
                                  int dtype, float eps, int64_t head_dim, int64_t gamma_head_stride,
                                  const qknorm_rope_t* rope, void* workspace, size_t workspace_bytes,
                                  void* stream);

/* Bytes of workspace that a backward call of these sizes needs (0 for sizes
 * it would reject; makes no HIP call). */
size_t qknorm_headwise_rope_backward_workspace(int64_t hq, int64_t hk, int64_t T, int dtype, int64_t head_dim,
                                               int64_t gamma_head_stride);

/* qknorm_headwise_rope_axes_backward -- gradients of qknorm_headwise_rope_axes, as
 * qknorm_headwise_rope_backward gives those of qknorm_headwise_rope (with its workspace). */
int qknorm_headwise_rope_axes_backward(const qknorm_grad_operand_t* q, const qknorm_grad_operand_t* k, int64_t T,
                                       int dtype, float eps, int64_t head_dim, int64_t gamma_head_stride,
                                       const qknorm_rope_t* rope, const qknorm_axes_t* axes, void* workspace,
                                       size_t workspace_bytes, void* stream);

typedef enum qknorm_cache_format {
  QKNORM_CACHE_ROWS = 0,  /* elements of the row type */
  QKNORM_CACHE_MXFP4 = 1, /* 4 bits an element: E2M1 codes (0 .5 1 1.5 2 3 4 6 and their negatives;
                             an even channel in its byte's low half) and one E8M0 scale byte (2^(byte - 127))
                             per 32 channels of a head. Written blocks take E = floor(log2(largest
                             magnitude)) - 2, held to [-100, 125], codes rounded to nearest even and
                             saturated at 6. A block that held an infinity or NaN gets the byte 255; bytes
                             above 252 read as NaN. */
  QKNORM_CACHE_MXFP8 = 3  /* 8 bits an element: E4M3 codes (bias 7, max 448, 0x7F and 0xFF NaN) and one E8M0
                             scale byte per 32 channels of a head. Written blocks take E = floor(log2(largest
                             magnitude)) - 8, held to [-100, 119], codes rounded to nearest even and
                             saturated at 448. A block that held an infinity or NaN gets the byte 255; bytes
                             above 246 read as NaN. */
} qknorm_cache_format_t;

/*
 * A paged cache of keys and values. Token `slot % page_size` of page `slot /
 * page_size` and key head h begins at
 *     k + page * page_stride + h * head_stride + token * token_stride
 * (elements of the row type, or bytes for MXFP4 and MXFP8), head_dim consecutive
 * elements (head_dim / 2 or head_dim bytes); its scales at
 *     k_scales + page * scale_page_stride + h * scale_head_stride + token * head_dim / 32
 * (bytes). v is laid out alike.
 */
typedef struct qknorm_cache {
  int format;              /* qknorm_cache_format_t */
  void* k;
  void* v;
  void* k_scales;          /* MXFP4 and MXFP8 only, as are the two strides below */
  void* v_scales;
  int64_t page_stride;     /* MXFP4, MXFP8: multiples of 16, and k and v 16-byte aligned */
  int64_t head_stride;
  int64_t token_stride;    /* MXFP4: head_dim / 2 (a head's tokens are packed); MXFP8: a multiple of 16 */
  int64_t scale_page_stride;   /* multiples of 16, and the scales 16-byte aligned */
  int64_t scale_head_stride;
  int64_t n_pages;         /* > 0 */
  int64_t page_size;       /* tokens, a power of two; MXFP4, MXFP8: at least 16 */
  int64_t heads;           /* key heads */
} qknorm_cache_t;

/*
 * qknorm_paged_append -- a step's keys and values into a paged cache, and its
 * queries made ready, in one pass over packed QKV rows: Q heads are
 * normalized and rotated into q->y, K heads normalized and rotated into the
 * cache, V heads taken as they are.
 *
 *   q      NULL: only K and V are appended. q->y as in qknorm_headwise_rope.
 *   k, v   k->h == v->h == cache->heads * head_dim. k->y and v->y may be NULL;
 *          otherwise they receive, as rows, the values the cache now holds.
 *   gamma  q->gamma or k->gamma NULL: that side is rotated but not normalized
 *          (for example after qknorm_fused). v->gamma is not used.
 *   slots  device int64 [T]: where each token goes (page * page_size + place in
 *          the page). A token whose slot is negative, or past the last page,
 *          is passed over: nothing of its row is written anywhere. No two
 *          tokens of a call may have the same slot (which of them, or which
 *          mixture, is kept would be undefined).
 *   dtype  QKNORM_F32 or QKNORM_BF16
 *   other arguments as for qknorm_headwise_rope.
 *
 * MXFP4 and MXFP8 need head_dim % 32 == 0. Keys bound for codes are formed in float32,
 * and again in float64 where a code or a scale is near a border, or a sum out
 * of float32's range, so that the codes are what exact arithmetic gives. No
 * other slot of the cache is written. Outputs and the cache must not overlap
 * each other or the inputs (q->y == q->x in place apart); k->y and v->y may not
 * be in place.
 */
int qknorm_paged_append(const qknorm_operand_t* q, const qknorm_operand_t* k, const qknorm_operand_t* v, int64_t T,
                        int dtype, float eps, int64_t head_dim, int64_t gamma_head_stride,
                        const qknorm_rope_t* rope, const qknorm_cache_t* cache, const int64_t* slots, void* stream);

/* qknorm_paged_append_axes -- qknorm_paged_append with positions on several axes
 * (axes as for qknorm_headwise_rope_axes). */
int qknorm_paged_append_axes(const qknorm_operand_t* q, const qknorm_operand_t* k, const qknorm_operand_t* v, int64_t T,
                             int dtype, float eps, int64_t head_dim, int64_t gamma_head_stride,
                             const qknorm_rope_t* rope, const qknorm_axes_t* axes, const qknorm_cache_t* cache,
                             const int64_t* slots, void* stream);

/*
 * qknorm_paged_gather -- reads a paged cache back: row t of k_rows and v_rows gets
 * the keys and values that slot slots[t] holds, heads side by side, in the row
 * type. The inverse of qknorm_paged_append for a prefix that is to be used
 * elsewhere (another layout, another device, an exact product).
 *
 *   cache   any format. QKNORM_CACHE_ROWS: elements of `dtype`, copied as they are.
 *   slots   device int64 [T], as in qknorm_paged_append: a negative slot, or one past
 *           the last page, leaves its row as it was. The same slot may occur more than
 *           once.
 *   dtype   QKNORM_F32 or QKNORM_BF16: the type of the rows written. Codes are widened
 *           exactly where their value fits it (bf16: all values of at least 2^-130, and below
 *           it multiples of 2^-133; others are rounded to nearest).
 *   k_rows, ld_k, v_rows, ld_v  row strides in elements, >= cache->heads * head_dim;
 *           one of them may be NULL (not wanted). They must not overlap each other or
 *           the cache.
 *   head_dim <= QKNORM_MAX_ROPE_HEAD, a multiple of 32 for MXFP4 and MXFP8.
 */
int qknorm_paged_gather(const qknorm_cache_t* cache, int64_t head_dim, const int64_t* slots, int64_t T, int dtype,
                        void* k_rows, int64_t ld_k, void* v_rows, int64_t ld_v, void* stream);

/* The batch that the attention calls work on. All arrays are device memory. */
typedef struct qknorm_batch {
  const int32_t* block_table;  /* [B][table_pages]: page ids in sequence order; row stride ld_table.
                                  An id outside [0, n_pages) among a sequence's tokens makes the rows
                                  that see them NaN. */
  int64_t ld_table;
  int64_t table_pages;
  const int32_t* seq_lens;     /* [B] cached tokens, those of this call's queries among them; held to
                                  [0, table_pages * page_size] */
  const int32_t* cu_q;         /* [B + 1] first query row of each sequence, increasing, the last one
                                  at most T; NULL: one query row per sequence (T == B). Rows outside
                                  every sequence are left as they were. */
  int64_t B;                   /* sequences, >= 0 */
  int64_t max_q;               /* most query rows and cached tokens of any sequence, as far as the */
  int64_t max_len;             /* caller knows (> 0): they shape the launch; larger ones stay correct */
} qknorm_batch_t;

/*
 * qknorm_paged_attend -- attention of T query rows over a paged MXFP4 cache:
 * out = softmax(scale q k^T + mask) v for each query head; head j reads key
 * head j / (query heads / key heads). Query i of the n of a sequence stands at
 * position seq_len - n + i and sees tokens up to its own (causal) or all
 * (causal == 0) of the sequence, and with window > 0 only tokens at positions
 * > its own - window. A row that sees nothing (an empty sequence, a position
 * below 0) is 0.
 *
 *   q          x, ld_x, y, ld_y (rows of q->h = query heads * head_dim); gamma is
 *              not used. 16-byte aligned, strides multiples of 8. y may not overlap x.
 *   dtype      QKNORM_BF16
 *   cache      format QKNORM_CACHE_MXFP4; the query heads are a multiple of cache->heads
 *   head_dim   64, 128 or 256
 *   scale      finite, > 0 (1/sqrt(head_dim) usually)
 *   workspace  at least qknorm_paged_attend_workspace(...) bytes, 16-byte aligned,
 *              not shared with a call that may run at the same time; its contents
 *              need no preparation. May be NULL where that size is 0.
 *
 * Scores, softmax statistics and sums are float32; probabilities are rounded
 * to bf16 for the second product, the result once more. Infinities and NaN of
 * cached tokens reach only the rows that see those tokens.
 */
int qknorm_paged_attend(const qknorm_operand_t* q, int64_t T, int dtype, const qknorm_cache_t* cache,
                        int64_t head_dim, const qknorm_batch_t* batch, float scale, int causal, int64_t window,
                        void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace that an attend call of these sizes needs, with any window
 * (0 for sizes it would reject; makes no HIP call). max_q is 1 for a call
 * without cu_q. */
size_t qknorm_paged_attend_workspace(int64_t T, int64_t heads_q, int64_t heads_k, int64_t head_dim, int64_t B,
                                     int64_t max_q, int64_t max_len);

/*
 * qknorm_paged_attend_wide -- qknorm_paged_attend over a cache of bf16 rows or
 * MXFP8: prompts, chunks of new tokens behind what the cache holds, and single
 * tokens.
 *
 *   cache      format QKNORM_CACHE_ROWS (of bf16) or QKNORM_CACHE_MXFP8; pages of at
 *              least 16 tokens; 16-byte aligned pointers, and page, head and token
 *              strides multiples of 16 bytes, a head's tokens less than 4 GiB / 16 apart
 *   workspace  at least qknorm_paged_attend_wide_workspace(...) bytes, as there
 *   other arguments as for qknorm_paged_attend.
 *
 * Scores, softmax statistics and sums are float32; probabilities are rounded to
 * bf16 for the second product (their sums are of the rounded ones), the result once
 * more. An infinity or NaN of a cached token reaches only the rows that see the
 * token: a NaN of K makes the whole row NaN, one of V its column; an infinite value
 * gives an infinity, or NaN where its probability vanishes in float32.
 */
int qknorm_paged_attend_wide(const qknorm_operand_t* q, int64_t T, int dtype, const qknorm_cache_t* cache,
                             int64_t head_dim, const qknorm_batch_t* batch, float scale, int causal, int64_t window,
                             void* workspace, size_t workspace_bytes, void* stream);

/* Bytes of workspace that such a call needs, with any window (0 for sizes it
 * would reject; makes no HIP call). max_q is 1 for a call without cu_q. */
size_t qknorm_paged_attend_wide_workspace(int64_t T, int64_t heads_q, int64_t heads_k, int64_t head_dim, int64_t B,
                                          int64_t max_q, int64_t max_len);

/* Message for the last non-OK return on the calling thread ("" if none). */
const char* qknorm_last_error(void);

/* QKNORM_ABI_VERSION of the built library. */
int qknorm_abi_version(void);

/*
 * qknorm_describe_plan -- writes a one-line description of the launch the
 * given call would make (element-wise or 16-byte path, lanes per shard,
 * chunks per lane, waves per token, and where they apply: token groups per
 * block, gamma held widened in registers, a cap on blocks per compute unit)
 * into buf (NUL-terminated, truncated to len). Validates like the call itself (op selects which one; `shards` is
 * ignored for QKNORM_OP_APPLY_WITH_STATS) and makes no HIP call, so it works
 * without a GPU. Device pointers are only compared, never dereferenced.
 */
int qknorm_describe_plan(int op, const qknorm_operand_t* q, const qknorm_operand_t* k,
                         int64_t T, int dtype, int shards, char* buf, size_t len);

/* As qknorm_describe_plan, for qknorm_headwise. */
int qknorm_describe_headwise_plan(const qknorm_operand_t* q, const qknorm_operand_t* k, int64_t T,
                                  int dtype, int64_t head_dim, int64_t gamma_head_stride, char* buf,
                                  size_t len);

#ifdef __cplusplus
}
#endif

#endif /* QKNORM_H */

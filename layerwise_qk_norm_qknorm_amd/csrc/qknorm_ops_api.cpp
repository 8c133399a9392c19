// C ABI of the operators around headwise QK-Norm: argument validation and
// planning for the norm with the rotation, its gradients, the paged append,
// reading a cache back and attention over it. Plain C++ with no HIP call, as
// qknorm_api.cpp; only the qkn::launch_* functions touch the HIP runtime.

#include <algorithm>
#include <cmath>
#include <cstring>
#include <string>
#include <utility>

#include "qknorm.h"
#include "qknorm_checks.hpp"
#include "qknorm_internal.hpp"
#include "qknorm_ops.hpp"

using namespace qkn;

namespace {

constexpr int64_t kMaxWidth = (int64_t)1 << 30;
constexpr int64_t kMaxTokens = (int64_t)1 << 30;          // of a sequence
constexpr int64_t kLaunchThreads = ((int64_t)1 << 32) - 1;   // of a launch

int log2_of(int64_t v) {
  int n = 0;
  while (((int64_t)1 << n) < v) ++n;
  return n;
}

bool power_of_two(int64_t v) { return v > 0 && (v & (v - 1)) == 0; }

bool multiple(const void* p, int64_t n) { return (uintptr_t)p % (uintptr_t)n == 0; }

Region bytes_of(const void* p, int64_t n) { return Region{(uintptr_t)p, n, n, n > 0 ? 1 : 0, 1}; }

// Alignments (bytes) that a piece size is held against.
struct Aligned {
  bool ok = true;
  void need(const void* p, int64_t n) { ok = ok && multiple(p, n); }
  void need(int64_t v, int64_t n) { ok = ok && v % n == 0; }
};

// Checks of the scalars and the rotation that the calls share.
int check_common(const char* fn, int64_t T, int dtype, bool fp8, float eps, int64_t head_dim, int64_t gstride,
                 const qknorm_rope_t* rope) {
  if (!elem_size(dtype)) return fail(QKNORM_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, dtype);
  if (dtype == QKNORM_FP8_E4M3 && !fp8)
    return fail(QKNORM_ERR_UNSUPPORTED, "%s: FP8 rows are not supported (float32 or bf16)", fn);
  if (T < 0) return fail(QKNORM_ERR_INVALID_ARG, "%s: T = %lld < 0", fn, (long long)T);
  if (!(std::isfinite(eps) && eps >= 0.0f)) return fail(QKNORM_ERR_INVALID_ARG, "%s: eps must be finite and >= 0", fn);
  if (head_dim <= 0) return fail(QKNORM_ERR_INVALID_ARG, "%s: head_dim = %lld", fn, (long long)head_dim);
  if (head_dim > kRopeMaxHead)
    return fail(QKNORM_ERR_UNSUPPORTED, "%s: head_dim = %lld > %d", fn, (long long)head_dim, kRopeMaxHead);
  if (gstride < 0 || gstride > kMaxWidth)
    return fail(QKNORM_ERR_INVALID_ARG, "%s: gamma_head_stride = %lld", fn, (long long)gstride);
  if (rope && rope->rot_dim) {
    if (rope->rot_dim < 0 || rope->rot_dim % 2 || rope->rot_dim > head_dim)
      return fail(QKNORM_ERR_INVALID_ARG, "%s: rot_dim = %lld is not an even number in [0, head_dim]", fn,
                  (long long)rope->rot_dim);
    if (rope->ld < rope->rot_dim) return fail(QKNORM_ERR_INVALID_ARG, "%s: rope->ld must be >= rot_dim", fn);
    if (rope->n_positions <= 0 || !fits(rope->n_positions, rope->ld, rope->rot_dim, 4))
      return fail(QKNORM_ERR_INVALID_ARG, "%s: rope->n_positions = %lld", fn, (long long)rope->n_positions);
    if (T > 0) {
      if (!rope->cos_sin || !rope->positions)
        return fail(QKNORM_ERR_INVALID_ARG, "%s: rope->cos_sin and positions are required", fn);
      if (!multiple(rope->cos_sin, 4) || !multiple(rope->positions, 8))
        return fail(QKNORM_ERR_INVALID_ARG, "%s: rope pointers must be aligned to their element size", fn);
    }
  }
  return QKNORM_OK;
}

// Positions on several axes, where there is a rotation.
int check_axes(const char* fn, const qknorm_rope_t* rope, const qknorm_axes_t* axes, int64_t T) {
  if (!axes || !rope || !rope->rot_dim) return QKNORM_OK;
  if (axes->n_axes < 1 || axes->n_axes > QKNORM_MAX_AXES)
    return fail(QKNORM_ERR_INVALID_ARG, "%s: n_axes = %d is not in [1, %d]", fn, axes->n_axes, QKNORM_MAX_AXES);
  if (!axes->axis) return fail(QKNORM_ERR_INVALID_ARG, "%s: axes->axis is required", fn);
  for (int64_t i = 0; i < rope->rot_dim / 2; ++i)
    if (axes->axis[i] >= axes->n_axes)
      return fail(QKNORM_ERR_INVALID_ARG, "%s: axis %d of angle %lld is not below n_axes = %d", fn, axes->axis[i],
                  (long long)i, axes->n_axes);
  if (axes->ld_positions < 0 || !fits(axes->n_axes, axes->ld_positions, T, 8))
    return fail(QKNORM_ERR_INVALID_ARG, "%s: ld_positions = %lld", fn, (long long)axes->ld_positions);
  return QKNORM_OK;
}

// What the kernels take of them.
void axes_args(const qknorm_rope_t* rope, const qknorm_axes_t* axes, RopeAxes* out) {
  if (!axes || !rope || !rope->rot_dim || axes->n_axes == 1) return;   // n == 0: one axis
  out->n = axes->n_axes;
  out->ld = axes->ld_positions;
  for (int64_t i = 0; i < rope->rot_dim / 2; ++i) out->of[i >> 4] |= (uint32_t)axes->axis[i] << (2 * (i & 15));
}

int check_width(const char* fn, const char* nm, int64_t h, int64_t head_dim) {
  if (h <= 0 || h % head_dim)
    return fail(QKNORM_ERR_INVALID_ARG, "%s: %s->h = %lld is not a positive multiple of head_dim %lld", fn, nm,
                (long long)h, (long long)head_dim);
  if (h > kMaxWidth) return fail(QKNORM_ERR_UNSUPPORTED, "%s: %s->h is too wide", fn, nm);
  return QKNORM_OK;
}

int check_rows(const char* fn, const char* what, const void* p, int64_t ld, int64_t h, int64_t T, int64_t esz) {
  if (ld < h) return fail(QKNORM_ERR_INVALID_ARG, "%s: %s row stride must be >= h", fn, what);
  if (T == 0) return QKNORM_OK;
  if (!p) return fail(QKNORM_ERR_INVALID_ARG, "%s: %s is required", fn, what);
  if (!multiple(p, esz))
    return fail(QKNORM_ERR_INVALID_ARG, "%s: %s must be aligned to its element size", fn, what);
  if (!fits(T, ld, h, esz)) return fail(QKNORM_ERR_INVALID_ARG, "%s: %s rows exceed the address range", fn, what);
  return QKNORM_OK;
}

// One 16-byte chunk of a head per lane, where chunks of the head and of half
// the rotation are powers of two; else the widest piece (16 bytes, 8 bytes, one
// element) that the shape allows. `aligned(bytes, angles)` answers for the
// addresses: rows at multiples of `bytes`, the table at those of `angles`
// elements.
template <class F>
RopePlan plan_pieces(int dtype, int64_t head_dim, int64_t rot, bool inter, F aligned) {
  RopePlan p;
  const int esz = row_elem_bytes(dtype);
  const int full = 16 / esz;
  if (head_dim % full == 0 && power_of_two(head_dim / full) && head_dim / full <= 64 &&
      (inter ? rot % full == 0 : rot == 0 || ((rot / 2) % full == 0 && power_of_two(rot / 2 / full))) &&
      aligned(16, inter ? full / 2 : full)) {
    p.whole = 1;
    p.piece_bytes = 16;
    p.vw = full;
    p.pairs = p.lanes = (int)(head_dim / full);
    return p;
  }
  for (int pb : {16, 8, esz}) {
    const int vw = pb / esz;
    if (vw > 1) {
      if (head_dim % (2 * vw) || (head_dim - rot) % (2 * vw) || rot % (2 * vw) || head_dim / (2 * vw) > 64) continue;
      if (!inter && (rot / 2) % vw) continue;
      if (!aligned(pb, vw)) continue;
    }
    p.piece_bytes = pb;
    p.vw = vw;
    p.pairs = (int)((head_dim + 2 * vw - 1) / (2 * vw));
    p.lanes = 1;
    while (p.lanes < p.pairs && p.lanes < 64) p.lanes *= 2;
    p.np = p.pairs > 64 ? 8 : 1;
    break;
  }
  return p;
}

int slots_of(int64_t heads, const RopePlan& p) { return (int)((heads * p.lanes + 63) / 64); }

// Slots per wave. Several share the token's angles and keep more loads in
// flight; calls of few tokens spread their slots over more waves. The waves of
// a side take whole numbers of slots, so of the counts tried the one that
// leaves fewest idle, of equals the largest (10 + 2 heads of 128, 16384
// tokens: three slots 24.1 us, two 26.3).
void plan_waves(RopePlan* p, const int (&slots)[3], int64_t T) {
  const int n = slots[0] + slots[1] + slots[2];
  const auto groups = [&](int s) { return (slots[0] + s - 1) / s + (slots[1] + s - 1) / s + (slots[2] + s - 1) / s; };
  p->slots = 1;
  if (p->whole) {
    if (T * n >= 8192) {
      int best = n;
      for (int s : {4, 3, 2})
        if (groups(s) * s - n < best) best = groups(s) * s - n, p->slots = s;
    }
    p->groups = groups(p->slots);
    return;
  }
  if (p->piece_bytes == 16 && T * n >= 4096) p->slots = 3;
  p->waves = (n + p->slots - 1) / p->slots;
  if (p->waves > kRopeMaxWaves) p->waves = kRopeMaxWaves;
  p->tokens = p->waves >= 4 ? 1 : 4 / p->waves;
}

void table_args(const qknorm_rope_t* rope, const RopePlan& p, int* rot, int* rot_pairs, const float** cs,
                int64_t* ld, int64_t* n, const int64_t** pos) {
  *rot = rope ? (int)rope->rot_dim : 0;
  *rot_pairs = *rot / (2 * p.vw);
  *cs = *rot ? rope->cos_sin : nullptr;
  *ld = *rot ? rope->ld : 0;
  *n = *rot ? rope->n_positions : 0;
  *pos = *rot ? rope->positions : nullptr;
}

bool table_aligned(const qknorm_rope_t* rope, int angles) {
  if (!rope || !rope->rot_dim) return true;
  const int64_t n = angles * 4 < 16 ? angles * 4 : 16;
  return multiple(rope->cos_sin, n) && rope->ld * 4 % n == 0 && rope->rot_dim / 2 * 4 % n == 0;
}

Region table_region(const qknorm_rope_t* rope) {
  if (!rope || !rope->rot_dim) return Region{0, 1, 0, 0, 1};
  return Region{(uintptr_t)rope->cos_sin, rope->ld, rope->rot_dim, rope->n_positions, 4};
}
Region positions_region(const qknorm_rope_t* rope, const qknorm_axes_t* axes, int64_t T) {
  if (!rope || !rope->rot_dim) return Region{0, 1, 0, 0, 1};
  return bytes_of(rope->positions, ((axes ? (axes->n_axes - 1) * axes->ld_positions : 0) + T) * 8);
}
Region gamma_region(const void* gamma, int64_t h, int64_t head_dim, int64_t gstride, int dtype) {
  return bytes_of(gamma, gamma ? ((h / head_dim - 1) * gstride + head_dim) * (int64_t)gamma_size(dtype) : 0);
}

// ------------------------------------------------------------ forward, append
struct RopeChecked {
  RopePlan plan;
  RopeAxesArgs args;
};

bool coded(const qknorm_cache_t* c) { return c->format != QKNORM_CACHE_ROWS; }
const char* format_name(const qknorm_cache_t* c) { return c->format == QKNORM_CACHE_MXFP4 ? "MXFP4" : "MXFP8"; }
// Elements of the row type, or bytes of codes, of a token's head.
int64_t held_row(const qknorm_cache_t* c, int64_t head_dim) {
  return c->format == QKNORM_CACHE_MXFP4 ? head_dim / 2 : head_dim;
}

int check_cache(const char* fn, const qknorm_cache_t* c, int64_t head_dim, int64_t esz, bool need_pointers) {
  if (!c) return fail(QKNORM_ERR_INVALID_ARG, "%s: a cache descriptor is required", fn);
  if (c->format != QKNORM_CACHE_ROWS && c->format != QKNORM_CACHE_MXFP4 && c->format != QKNORM_CACHE_MXFP8)
    return fail(QKNORM_ERR_INVALID_ARG, "%s: unknown cache format %d", fn, c->format);
  const bool codes = coded(c);
  if (c->heads <= 0 || c->heads > kMaxWidth / head_dim)
    return fail(QKNORM_ERR_INVALID_ARG, "%s: cache->heads = %lld", fn, (long long)c->heads);
  if (c->n_pages <= 0 || !power_of_two(c->page_size) || c->page_size > ((int64_t)1 << 30))
    return fail(QKNORM_ERR_INVALID_ARG, "%s: the cache needs pages, and a power of two of tokens in each", fn);
  if (codes && head_dim % 32)
    return fail(QKNORM_ERR_INVALID_ARG, "%s: head_dim = %lld is not a multiple of 32 (%s)", fn, (long long)head_dim,
                format_name(c));
  if (codes && c->page_size < 16)
    return fail(QKNORM_ERR_INVALID_ARG, "%s: %s pages hold at least 16 tokens", fn, format_name(c));
  const int64_t row = held_row(c, head_dim);
  if (c->token_stride < row || c->head_stride < row || c->page_stride < row)
    return fail(QKNORM_ERR_INVALID_ARG, "%s: cache strides must hold a token's head", fn);
  // positions of all tokens in a page and head, of all heads, of all pages: byte ranges that fit
  const int64_t unit = codes ? 1 : esz;
  const int64_t lim = INT64_MAX / 4 / unit;
  if (c->token_stride > lim / c->page_size || c->head_stride > lim / c->heads || c->page_stride > lim / c->n_pages)
    return fail(QKNORM_ERR_INVALID_ARG, "%s: the cache exceeds the address range", fn);
  if (c->n_pages > lim / c->page_size)
    return fail(QKNORM_ERR_INVALID_ARG, "%s: the cache has too many tokens", fn);
  if (codes) {
    if (c->format == QKNORM_CACHE_MXFP4 && c->token_stride != head_dim / 2)
      return fail(QKNORM_ERR_INVALID_ARG, "%s: MXFP4 tokens of a head are packed (token_stride = head_dim / 2)", fn);
    const int64_t srow = head_dim / 32;
    if (c->scale_page_stride < srow || c->scale_head_stride < srow || c->scale_page_stride > lim / c->n_pages ||
        c->scale_head_stride > lim / c->heads)
      return fail(QKNORM_ERR_INVALID_ARG, "%s: scale strides must hold a token's scales", fn);
    if (c->page_stride % 16 || c->head_stride % 16 || c->scale_page_stride % 16 || c->scale_head_stride % 16)
      return fail(QKNORM_ERR_INVALID_ARG, "%s: %s page and head strides must be multiples of 16 bytes", fn,
                  format_name(c));
    if (c->token_stride % 16)
      return fail(QKNORM_ERR_INVALID_ARG, "%s: %s token strides must be multiples of 16 bytes", fn, format_name(c));
  }
  if (!need_pointers) return QKNORM_OK;
  if (!c->k || !c->v || (codes && (!c->k_scales || !c->v_scales)))
    return fail(QKNORM_ERR_INVALID_ARG, "%s: cache pointers are required", fn);
  if (codes && !(multiple(c->k, 16) && multiple(c->v, 16) && multiple(c->k_scales, 16) && multiple(c->v_scales, 16)))
    return fail(QKNORM_ERR_INVALID_ARG, "%s: %s cache pointers must be 16-byte aligned", fn, format_name(c));
  if (!codes && !(multiple(c->k, esz) && multiple(c->v, esz)))
    return fail(QKNORM_ERR_INVALID_ARG, "%s: cache pointers must be aligned to their element size", fn);
  return QKNORM_OK;
}

// One of the cache's arrays: a row of bytes per page where pages are the
// outermost axis (so that arrays which take turns within one allocation's pages
// are told apart), the whole span otherwise.
Region cache_region(const qknorm_cache_t* c, const void* p, bool scales, int64_t head_dim, int64_t esz) {
  const int64_t unit = coded(c) ? 1 : esz, row = held_row(c, head_dim);
  const int64_t inner =
      scales ? (c->heads - 1) * c->scale_head_stride + c->page_size * (head_dim / 32)
             : ((c->heads - 1) * c->head_stride + (c->page_size - 1) * c->token_stride + row) * unit;
  const int64_t page = scales ? c->scale_page_stride : c->page_stride * unit;
  if (inner <= page) return Region{(uintptr_t)p, page, inner, c->n_pages, 1};
  return bytes_of(p, (c->n_pages - 1) * page + inner);
}

// True if the cache's two largest strides keep heads and tokens of one page,
// and pages, apart: any nesting order of (page, head, token) with every stride
// at least as large as what lies inside it.
bool cache_nests(const qknorm_cache_t* c, int64_t head_dim) {
  struct Axis {
    int64_t stride, n;
  };
  Axis ax[3] = {{c->page_stride, c->n_pages}, {c->head_stride, c->heads}, {c->token_stride, c->page_size}};
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2 - i; ++j)
      if (ax[j].stride > ax[j + 1].stride) std::swap(ax[j], ax[j + 1]);
  int64_t inner = held_row(c, head_dim);
  for (const Axis& x : ax) {
    if (x.n == 1) continue;
    if (x.stride < inner) return false;
    inner = x.stride * (x.n - 1) + inner;
  }
  if (!coded(c)) return true;
  const int64_t page = c->page_size * (head_dim / 32);
  const int64_t lo = c->scale_head_stride < c->scale_page_stride ? c->scale_head_stride : c->scale_page_stride;
  const bool head_inner = c->scale_head_stride <= c->scale_page_stride;
  const int64_t n_in = head_inner ? c->heads : c->n_pages, n_out = head_inner ? c->n_pages : c->heads;
  const int64_t hi = head_inner ? c->scale_page_stride : c->scale_head_stride;
  if (n_in > 1 && lo < page) return false;
  return n_out == 1 || hi >= (n_in > 1 ? lo * (n_in - 1) : 0) + page;
}

// Forward (v, cache and slots NULL) and append.
int check_rope(const char* fn, const qknorm_operand_t* q, const qknorm_operand_t* k, const qknorm_operand_t* v,
               int64_t T, int dtype, float eps, int64_t head_dim, int64_t gstride, const qknorm_rope_t* rope,
               const qknorm_axes_t* axes, const qknorm_cache_t* cache, const int64_t* slots, bool append,
               RopeChecked* out, bool* noop) {
  *noop = false;
  if (!k || (!append && !q) || (append && !v))
    return fail(QKNORM_ERR_INVALID_ARG, "%s: operand descriptors are required", fn);
  int rc = check_common(fn, T, dtype, !append, eps, head_dim, gstride, rope);
  if (rc || (rc = check_axes(fn, rope, axes, T))) return rc;
  const int64_t esz = (int64_t)elem_size(dtype), gsz = (int64_t)gamma_size(dtype);
  const qknorm_operand_t* ops[3] = {q, k, v};
  const char* nm[3] = {"q", "k", "v"};
  const char* xn[3] = {"q->x", "k->x", "v->x"};
  const char* yn[3] = {"q->y", "k->y", "v->y"};
  for (int c = 0; c < 3; ++c) {
    const qknorm_operand_t* o = ops[c];
    if (!o) continue;
    if ((rc = check_width(fn, nm[c], o->h, head_dim))) return rc;
    if ((rc = check_rows(fn, xn[c], o->x, o->ld_x, o->h, T, esz))) return rc;
    if (!append || c == 0 || o->y)
      if ((rc = check_rows(fn, yn[c], o->y, o->ld_y, o->h, T, esz))) return rc;
    if (!append && T > 0 && !o->gamma) return fail(QKNORM_ERR_INVALID_ARG, "%s: %s->gamma is required", fn, nm[c]);
    if (c < 2 && o->gamma && !multiple(o->gamma, gsz))
      return fail(QKNORM_ERR_INVALID_ARG, "%s: %s->gamma must be aligned to its element size", fn, nm[c]);
  }
  const bool codes = append && cache && coded(cache);
  if (append) {
    if ((rc = check_cache(fn, cache, head_dim, esz, T > 0))) return rc;
    if (k->h != cache->heads * head_dim || v->h != k->h)
      return fail(QKNORM_ERR_INVALID_ARG, "%s: k->h and v->h must be cache->heads * head_dim", fn);
    if (!cache_nests(cache, head_dim))
      return fail(QKNORM_ERR_INVALID_ARG, "%s: cache strides make tokens overlap", fn);
    if (T > 0 && (!slots || !multiple(slots, 8)))
      return fail(QKNORM_ERR_INVALID_ARG, "%s: slots must be an 8-byte aligned device pointer", fn);
  }
  if (T == 0) {
    *noop = true;
    return ok();
  }

  // Everything written against everything else.
  struct Buf {
    Region r;
    const char* name;
  };
  Buf outs[7], ins[12];
  int n_out = 0, n_in = 0;
  for (int c = 0; c < 3; ++c) {
    const qknorm_operand_t* o = ops[c];
    if (!o) continue;
    ins[n_in++] = {Region{(uintptr_t)o->x, o->ld_x, o->h, T, esz}, xn[c]};
    if (o->y) outs[n_out++] = {Region{(uintptr_t)o->y, o->ld_y, o->h, T, esz}, yn[c]};
    if (c < 2 && o->gamma) ins[n_in++] = {gamma_region(o->gamma, o->h, head_dim, gstride, dtype), "gamma"};
  }
  ins[n_in++] = {table_region(rope), "the rope table"};
  ins[n_in++] = {positions_region(rope, axes, T), "positions"};
  if (append) {
    ins[n_in++] = {bytes_of(slots, T * 8), "slots"};
    outs[n_out++] = {cache_region(cache, cache->k, false, head_dim, esz), "the k cache"};
    outs[n_out++] = {cache_region(cache, cache->v, false, head_dim, esz), "the v cache"};
    if (codes) {
      outs[n_out++] = {cache_region(cache, cache->k_scales, true, head_dim, esz), "the k scales"};
      outs[n_out++] = {cache_region(cache, cache->v_scales, true, head_dim, esz), "the v scales"};
    }
  }
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < i; ++j)
      if (may_overlap(outs[i].r, outs[j].r))
        return fail(QKNORM_ERR_INVALID_ARG, "%s: %s overlaps %s", fn, outs[i].name, outs[j].name);
    for (int j = 0; j < n_in; ++j) {
      const bool own = outs[i].name[0] == ins[j].name[0] && outs[i].name[1] == '-' && ins[j].name[1] == '-';
      if (own && same_region(outs[i].r, ins[j].r) && (!append || outs[i].name[0] == 'q')) continue;   // in place
      if (may_overlap(outs[i].r, ins[j].r))
        return fail(QKNORM_ERR_INVALID_ARG, "%s: %s overlaps %s", fn, outs[i].name, ins[j].name);
    }
  }

  const int64_t rot = rope ? rope->rot_dim : 0;
  const bool inter = rot && rope->interleaved;
  out->plan = plan_pieces(dtype, head_dim, rot, inter, [&](int pb, int angles) {
    Aligned al;
    const int vw = pb / (int)esz;
    for (const qknorm_operand_t* o : ops) {
      if (!o) continue;
      al.need(o->x, pb);
      al.need(o->ld_x * esz, pb);
      if (o->y && !(codes && o != q && pb < 16)) {
        al.need(o->y, pb);
        al.need(o->ld_y * esz, pb);
      }
      if (o->gamma && o != v) {
        const int64_t g = vw * gsz < 16 ? vw * gsz : 16;
        al.need(o->gamma, g);
        al.need(gstride * gsz, g);
      }
    }
    if (append && !codes) {
      al.need(cache->k, pb);
      al.need(cache->v, pb);
      al.need(cache->page_stride * esz, pb);
      al.need(cache->head_stride * esz, pb);
      al.need(cache->token_stride * esz, pb);
    }
    return al.ok && table_aligned(rope, angles);
  });
  RopePlan& p = out->plan;
  RopeAxesArgs& a = out->args;
  a = RopeAxesArgs{};
  int slots_in[3] = {0, 0, 0};
  for (int c = 0; c < 3; ++c) {
    const qknorm_operand_t* o = ops[c];
    if (!o) continue;
    a.side[c] = RopeSide{o->x, o->y, c < 2 ? o->gamma : nullptr, o->ld_x, o->ld_y, (int)(o->h / head_dim)};
    slots_in[c] = slots_of(a.side[c].heads, p);
  }
  plan_waves(&p, slots_in, T);
  if (!p.whole && slots_in[0] + slots_in[1] + slots_in[2] > 65535)
    return fail(QKNORM_ERR_UNSUPPORTED, "%s: too many heads", fn);
  p.apart = codes && q && p.whole && p.slots > 1;
  a.n_slots = slots_in[0] + slots_in[1] + slots_in[2];
  const int unit = p.whole ? p.slots : 1;   // sides begin at whole waves, or at slots
  a.first[1] = (slots_in[0] + unit - 1) / unit;
  a.first[2] = a.first[1] + (slots_in[1] + unit - 1) / unit;
  a.T = T;
  a.gstride = gstride;
  a.head_dim = (int)head_dim;
  a.pairs = p.pairs;
  table_args(rope, p, &a.rot, &a.rot_pairs, &a.cos_sin, &a.ld_table, &a.n_positions, &a.positions);
  axes_args(rope, axes, &a.axes);
  a.log2_lanes = log2_of(p.lanes);
  a.half_lanes = rot && !inter ? (int)(rot / 2 / p.vw) : 0;
  a.idle = p.lanes * p.np * 2 * p.vw != head_dim;
  a.waves = p.waves;
  a.tokens = p.tokens;
  a.waves_inv = (uint32_t)((65536 + p.waves - 1) / p.waves);
  a.inv_div = (float)(1.0 / (double)head_dim);
  a.eps = eps;
  if (append) {
    const int64_t unit = codes ? 1 : esz;
    a.slots = slots;
    a.n_tokens_held = cache->n_pages * cache->page_size;
    a.log2_page = log2_of(cache->page_size);
    a.cache[0] = (char*)cache->k;
    a.cache[1] = (char*)cache->v;
    a.scales[0] = (char*)cache->k_scales;
    a.scales[1] = (char*)cache->v_scales;
    a.page_stride = cache->page_stride * unit;
    a.head_stride = cache->head_stride * unit;
    a.token_stride = cache->token_stride * unit;
    a.scale_page_stride = cache->scale_page_stride;
    a.scale_head_stride = cache->scale_head_stride;
    a.y_wide = 1;
    for (int c = 1; c < 3; ++c)
      if (ops[c]->y && !(multiple(ops[c]->y, 16) && ops[c]->ld_y * esz % 16 == 0)) a.y_wide = 0;
  }
  return QKNORM_OK;
}

// ------------------------------------------------------------------ backward
// Blocks per slot of heads: as many as the chip holds at once over all slots
// (256 compute units of four, or three in the paired layout, whose kernels need
// more registers), never a few more, which would run alone. In eights, so that
// the blocks of all slots that take the same tokens run on one XCD, whose L2
// then holds those tokens' angles. bf16, 8192 tokens, heads of 128: 36 heads
// 45.8 us, 50.0 with 768 blocks, 47.6 with 1024 not in eights; 48 heads 59.7,
// 59.2, 60.0, and 82.8 with 8 blocks more than fit; float32, 32 heads 72.7, 77.5
// with 768.
int grad_workers(int n_slots, int64_t T, bool whole) {
  int64_t w = (whole ? 1024 : 768) / n_slots;
  if (w > 8) w -= w % 8;
  return (int)std::clamp<int64_t>(w, 1, (T + kGradWaves - 1) / kGradWaves);
}

// The layout the backward call takes at its widest workspace: rows depend on
// the piece size only through the slot count, which is largest for one element
// per piece.
size_t grad_workspace(int64_t heads_q, int64_t heads_k, int64_t T, int dtype, int64_t head_dim, int64_t gstride) {
  size_t most = 0;
  const int esz = row_elem_bytes(dtype);
  for (int pb : {32, 16, 8, esz}) {   // 32: one 16-byte chunk per lane, half a pair
    const int vw = pb == 32 ? 8 / esz : pb / esz;
    RopePlan p;
    p.pairs = (int)((head_dim + 2 * vw - 1) / (2 * vw));
    p.lanes = 1;
    while (p.lanes < p.pairs && p.lanes < 64) p.lanes *= 2;
    const int n = slots_of(heads_q, p) + slots_of(heads_k, p);
    const int64_t rows = (gstride == 0 ? n : heads_q + heads_k) * (int64_t)grad_workers(n, T, pb == 32);
    const size_t bytes = (size_t)rows * (size_t)head_dim * 4;
    if (bytes > most) most = bytes;
  }
  return most;
}

int check_grad(const char* fn, const qknorm_grad_operand_t* q, const qknorm_grad_operand_t* k, int64_t T, int dtype,
               float eps, int64_t head_dim, int64_t gstride, const qknorm_rope_t* rope, const qknorm_axes_t* axes,
               void* ws, size_t ws_bytes, RopePlan* plan, RopeGradAxesArgs* args, bool* noop) {
  *noop = false;
  if (!q || !k) return fail(QKNORM_ERR_INVALID_ARG, "%s: q and k operand descriptors are required", fn);
  int rc = check_common(fn, T, dtype, false, eps, head_dim, gstride, rope);
  if (rc || (rc = check_axes(fn, rope, axes, T))) return rc;
  if (gstride && gstride < head_dim)
    return fail(QKNORM_ERR_INVALID_ARG, "%s: gamma_head_stride = %lld is neither 0 nor >= head_dim", fn,
                (long long)gstride);
  const int64_t esz = (int64_t)elem_size(dtype), gsz = (int64_t)gamma_size(dtype);
  const qknorm_grad_operand_t* ops[2] = {q, k};
  const char* nm[2] = {"q", "k"};
  const char* names[2][3] = {{"q->x", "q->dy", "q->dx"}, {"k->x", "k->dy", "k->dx"}};
  for (int c = 0; c < 2; ++c) {
    const qknorm_grad_operand_t* o = ops[c];
    if ((rc = check_width(fn, nm[c], o->h, head_dim))) return rc;
    if ((rc = check_rows(fn, names[c][0], o->x, o->ld_x, o->h, T, esz))) return rc;
    if ((rc = check_rows(fn, names[c][1], o->dy, o->ld_dy, o->h, T, esz))) return rc;
    if ((rc = check_rows(fn, names[c][2], o->dx, o->ld_dx, o->h, T, esz))) return rc;
    if (T > 0 && (!o->gamma || !multiple(o->gamma, gsz)))
      return fail(QKNORM_ERR_INVALID_ARG, "%s: %s->gamma is required, aligned to its element size", fn, nm[c]);
    if (!multiple(o->dgamma, 4))
      return fail(QKNORM_ERR_INVALID_ARG, "%s: %s->dgamma must be aligned to 4 bytes", fn, nm[c]);
  }
  if (T == 0) {
    *noop = true;
    return ok();
  }
  const bool wanted = q->dgamma || k->dgamma;
  const size_t need = grad_workspace(q->h / head_dim, k->h / head_dim, T, dtype, head_dim, gstride);
  if (wanted && (!ws || !multiple(ws, 16) || ws_bytes < need))
    return fail(QKNORM_ERR_INVALID_ARG, "%s: the workspace must be 16-byte aligned, at least %zu bytes", fn, need);

  const auto rows = [&](const void* p, int64_t ld, int64_t h) { return Region{(uintptr_t)p, ld, h, T, esz}; };
  Region outs[5], ins[8];
  int n_out = 0, n_in = 0;
  for (int c = 0; c < 2; ++c) {
    const qknorm_grad_operand_t* o = ops[c];
    outs[n_out++] = rows(o->dx, o->ld_dx, o->h);
    ins[n_in++] = rows(o->x, o->ld_x, o->h);
    ins[n_in++] = rows(o->dy, o->ld_dy, o->h);
    ins[n_in++] = gamma_region(o->gamma, o->h, head_dim, gstride, dtype);
  }
  ins[n_in++] = table_region(rope);
  ins[n_in++] = positions_region(rope, axes, T);
  for (int c = 0; c < 2; ++c)
    if (ops[c]->dgamma) outs[n_out++] = gamma_region(ops[c]->dgamma, ops[c]->h, head_dim, gstride, QKNORM_F32);
  if (wanted) outs[n_out++] = bytes_of(ws, (int64_t)need);
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < i; ++j)
      if (may_overlap(outs[i], outs[j])) return fail(QKNORM_ERR_INVALID_ARG, "%s: outputs or workspace overlap", fn);
    for (int j = 0; j < n_in; ++j) {
      const bool own = i < 2 && j / 3 == i && j % 3 < 2;   // dx in place of its own x or dy
      if (own && same_region(outs[i], ins[j])) continue;
      if (may_overlap(outs[i], ins[j])) return fail(QKNORM_ERR_INVALID_ARG, "%s: an output overlaps an input", fn);
    }
  }

  const int64_t rot = rope ? rope->rot_dim : 0;
  *plan = plan_pieces(dtype, head_dim, rot, rot && rope->interleaved, [&](int pb, int angles) {
    Aligned al;
    const int vw = pb / (int)esz;
    for (const qknorm_grad_operand_t* o : ops) {
      al.need(o->x, pb);
      al.need(o->ld_x * esz, pb);
      al.need(o->dy, pb);
      al.need(o->ld_dy * esz, pb);
      al.need(o->dx, pb);
      al.need(o->ld_dx * esz, pb);
      const int64_t g = vw * gsz < 16 ? vw * gsz : 16;
      al.need(o->gamma, g);
      al.need(gstride * gsz, g);
    }
    return al.ok && table_aligned(rope, angles);
  });
  RopeGradAxesArgs& a = *args;
  a = RopeGradAxesArgs{};
  for (int c = 0; c < 2; ++c) {
    const qknorm_grad_operand_t* o = ops[c];
    a.first[c] = a.n_slots;
    a.side[c] = RopeGradSide{o->x, o->dy, o->dx, o->gamma, o->dgamma, o->ld_x, o->ld_dy, o->ld_dx,
                             (int)(o->h / head_dim)};
    a.n_slots += slots_of(a.side[c].heads, *plan);
  }
  if (a.n_slots > 65535 || (gstride && (wanted ? a.side[0].heads + a.side[1].heads : 0) > 65535))
    return fail(QKNORM_ERR_UNSUPPORTED, "%s: too many heads", fn);
  a.T = T;
  a.gstride = gstride;
  a.head_dim = (int)head_dim;
  a.pairs = plan->pairs;
  table_args(rope, *plan, &a.rot, &a.rot_pairs, &a.cos_sin, &a.ld_table, &a.n_positions, &a.positions);
  axes_args(rope, axes, &a.axes);
  a.log2_lanes = log2_of(plan->lanes);
  a.half_lanes = rot && !rope->interleaved ? (int)(rot / 2 / plan->vw) : 0;
  a.idle = plan->lanes * plan->np * 2 * plan->vw != head_dim;
  a.workers = grad_workers(a.n_slots, T, plan->whole);
  a.inv_div = (float)(1.0 / (double)head_dim);
  a.eps = eps;
  a.partial = (float*)ws;
  if (wanted && (size_t)rope_grad_rows(a) * (size_t)head_dim * 4 > need)
    return fail(QKNORM_ERR_UNSUPPORTED, "%s: the plan exceeds its workspace", fn);   // not reached: need covers every plan
  return QKNORM_OK;
}

// -------------------------------------------------------------------- attend
// Row tiles per block and the cache's split. Rows of a sequence beyond 16 and
// 32 take two and four row tiles (at most two at 256 columns), so that what
// is read and widened of the cache serves more rows.
//
// The cache is split so that the blocks fill one or two whole rounds of what
// the chip holds at once (256 compute units of three or two blocks, as in the
// kernel's launch bounds), whichever takes fewer steps of 128 tokens; a
// block's start and end count as two steps, the joining launch as four.
// Against splitting until there are about 1024 blocks (5 or 4 query heads to
// a key head, 8 key heads of 128 columns): one sequence of 65536 tokens 25.5
// -> 23.1 us, 64 of up to 8192 98 -> 90, 96 of 512 21.6 -> 11.7, 32 of 2048
// 21.1 -> 18.0; 32 of 4096 with 4 key heads of 256 columns 35.8 -> 30.6.
constexpr int64_t kRounds = 2, kBlockSteps = 2, kJoinSteps = 4;

// Blocks along the rows are meant for max_q rows of each sequence, and those
// of shorter ones end at once, which costs 0.55 ns each. Where that asks for
// more than 2^17 blocks (max_q left at T, or one long prompt among many
// tokens) a sequence gets as many as fill the chip by themselves, or four
// times its even share of the row tiles there are, and they loop over its
// rows. 40 over 8 heads of 128: 512 sequences of 1 to 64 rows on 512 tokens,
// max_q left at T, 3575 us -> 738 (605 with max_q = 64); 256 of 64 to 170 rows
// 3314 -> 687 (629 with max_q = 170); 4096 rows and 511 of one row 1614 -> 1078;
// 8192 rows and 63 of one row 2986 -> 2899, and 3174 had they been held to what
// fills the chip there too.
constexpr int64_t kManyBlocks = (int64_t)1 << 17;
int64_t row_tiles_of(int64_t tiles, int64_t tile, int64_t heads_k, int64_t group, int64_t B, int64_t T,
                     int64_t resident) {
  const int64_t pairs = B * heads_k;
  const int64_t fill = std::max((resident + heads_k - 1) / heads_k, kManyBlocks / pairs);
  const int64_t even = 4 * (std::min(T, kMaxTokens) * group / tile + B) / B;
  const int64_t most = std::max(std::min(fill, kLaunchThreads / 256 / pairs), even);
  return std::min({tiles, most, (int64_t)65536});
}
//
// parts_per_step: bytes of partial results that are written and read again in the
// time of a step (0: not counted).
void split_cache(AttendPlan* p, int64_t blocks, int64_t resident, int64_t group, int64_t max_len, int64_t window,
                 int64_t part_bytes, int64_t parts_per_step) {
  const auto most = [&](int64_t len) { return std::max<int64_t>(1, std::min((len + 255) / 256, kRounds * resident / blocks)); };
  p->most_splits = (int)most(max_len);
  // what a block's rows see together, at most
  const int64_t span = window && window < max_len ? std::min(max_len, window + 16 * p->row_tile / group + 33) : max_len;
  const int64_t m = most(span);
  int64_t least = INT64_MAX;
  for (int64_t rounds = 0; rounds <= kRounds; ++rounds) {
    const int64_t s = std::clamp<int64_t>(rounds * resident / blocks, 1, m);
    int64_t chunk = ((span + s - 1) / s + 127) / 128 * 128;
    if (chunk < 256) chunk = 256;
    const int64_t n = (span + chunk - 1) / chunk;
    int64_t cost = (blocks * n + resident - 1) / resident * (chunk / 128 + kBlockSteps);
    if (n > 1) cost += kJoinSteps + (parts_per_step ? (int64_t)((double)n * (double)part_bytes / (double)parts_per_step) : 0);
    if (cost < least) least = cost, p->splits = (int)n, p->chunk = (int)chunk;
  }
}

AttendPlan plan_attend(int64_t head_dim, int64_t heads_k, int64_t group, int64_t B, int64_t T, int64_t max_q,
                       int64_t max_len, int64_t window) {
  AttendPlan p;
  p.head_dim = (int)head_dim;
  const int64_t rows = max_q * group;
  p.row_tile = rows <= 16 ? 1 : rows <= 32 || head_dim == 256 ? 2 : 4;
  const int64_t tiles = (rows + 16 * p.row_tile - 1) / (16 * p.row_tile);
  const int64_t resident = 256 * (p.row_tile * head_dim <= 128 ? 3 : 2);
  p.row_tiles = (int)row_tiles_of(tiles, 16 * p.row_tile, heads_k, group, B, T, resident);
  p.max_q = max_q;
  split_cache(&p, B * heads_k * p.row_tiles, resident, group, max_len, window, 0, 0);
  return p;
}

// The same for caches of rows and MXFP8. Up to 32 rows of a sequence (of a key head)
// share a block's four waves, which take the cache's tokens in turn; beyond them
// each wave takes 32 rows, four waves to a block, and eight from 129 rows on at 128
// columns, so that a staged tile serves 256 rows (4 x 531 .. 1024 rows x 5 heads on
// 4215 .. 8192 tokens: 422 us with four, 371 with eight; at 64 columns four waves at
// three blocks a unit are faster, 208 us against 213, at 256 their registers do not
// suffice). 257 to 384 rows take four again, which leave no third of the blocks'
// rows empty (4 x up to 64 rows x 5 heads on those tokens 78 us against 90; from 385
// on eight are as fast or faster).
//
// Up to 32 rows over a cache of rows are split for one block a compute unit, not the
// two that it holds: its four waves keep enough loads in flight, and fewer splits are
// joined (single tokens of 40 over 8 heads, 4 x 32768: 79.4 -> 68.4 us, 8 x 8192
// 45.6 -> 41.4, 1 x 65536 54.1 -> 52.3, 16 x 1000 17.5 -> 15.4). From MXFP8, whose
// loads are half as many bytes, 4 x 32768 would take 50.5 for 44.4. Workspaces are
// sized for two.
//
// A step of the kernel for more rows takes 4.6 us, in which 18 MB of partial results go to memory
// and back: 1024 rows x 5 heads on 4096 tokens, 160 blocks, are 117 to 123 us unsplit (from card
// to card) and 144 in three parts. Both are measured at 128 columns and taken for the other widths.
AttendPlan plan_attend_wide(bool codes, int64_t head_dim, int64_t heads_k, int64_t group, int64_t B, int64_t T,
                            int64_t max_q, int64_t max_len, int64_t window) {
  AttendPlan p;
  p.head_dim = (int)head_dim;
  const int64_t rows = max_q * group;
  const bool four = rows <= 128 || (rows > 256 && rows <= 384) || head_dim != 128;
  p.row_tile = rows <= 16 ? 1 : rows <= 32 ? 2 : four ? 8 : 16;
  const int64_t tiles = (rows + 16 * p.row_tile - 1) / (16 * p.row_tile);
  const int64_t resident = 256 * (head_dim == 256 || p.row_tile == 16 || (!codes && p.row_tile <= 2) ? 1
                                : head_dim == 64 && p.row_tile == 8                               ? 3
                                                                                                  : 2);
  p.row_tiles = (int)row_tiles_of(tiles, 16 * p.row_tile, heads_k, group, B, T, resident);
  p.max_q = max_q;
  split_cache(&p, B * heads_k * p.row_tiles, resident, group, max_len, window, T * heads_k * group * (head_dim + 2) * 8,
              p.row_tile >= 8 ? 18 * 1000 * 1000 : 0);
  return p;
}

bool attend_sizes_ok(int64_t T, int64_t heads_q, int64_t heads_k, int64_t head_dim, int64_t B, int64_t max_q,
                     int64_t max_len) {
  return T >= 0 && heads_k > 0 && heads_q > 0 && heads_q % heads_k == 0 && heads_q <= 65536 &&
         (head_dim == 64 || head_dim == 128 || head_dim == 256) && B >= 0 && B <= ((int64_t)1 << 20) && max_q > 0 &&
         max_q <= kMaxTokens && max_len > 0 && max_len <= kMaxTokens;
}

// Query rows whose numbers, with all heads of a group side by side, keep clear of 32 bits.
bool attend_rows_ok(int64_t T, int64_t group) { return T <= kMaxTokens / 4 / group; }

size_t attend_workspace(const AttendPlan& p, int64_t T, int64_t heads_q) {
  if (p.most_splits <= 1) return 0;
  return (size_t)T * (size_t)heads_q * (size_t)p.most_splits * (size_t)(p.head_dim + 2) * 4;
}

int rope_forward(const char* fn, const qknorm_operand_t* q, const qknorm_operand_t* k, int64_t T, int dtype, float eps,
                 int64_t head_dim, int64_t gstride, const qknorm_rope_t* rope, const qknorm_axes_t* axes,
                 void* stream) {
  RopeChecked c;
  bool noop;
  const int rc = check_rope(fn, q, k, nullptr, T, dtype, eps, head_dim, gstride, rope, axes, nullptr, nullptr, false,
                            &c, &noop);
  if (rc || noop) return rc;
  std::string err;
  if (launch_rope(ROPE_FORWARD, dtype, c.args.rot && rope->interleaved, c.plan, c.args, stream, &err))
    return fail(QKNORM_ERR_HIP, "%s: %s", fn, err.c_str());
  return ok();
}

int rope_backward(const char* fn, const qknorm_grad_operand_t* q, const qknorm_grad_operand_t* k, int64_t T, int dtype,
                  float eps, int64_t head_dim, int64_t gstride, const qknorm_rope_t* rope, const qknorm_axes_t* axes,
                  void* workspace, size_t workspace_bytes, void* stream) {
  RopePlan plan;
  RopeGradAxesArgs args;
  bool noop;
  const int rc = check_grad(fn, q, k, T, dtype, eps, head_dim, gstride, rope, axes, workspace, workspace_bytes, &plan,
                            &args, &noop);
  if (rc || noop) return rc;
  std::string err;
  if (launch_rope_grad(dtype, args.rot && rope->interleaved, plan, args, stream, &err))
    return fail(QKNORM_ERR_HIP, "%s: %s", fn, err.c_str());
  return ok();
}

int append(const char* fn, const qknorm_operand_t* q, const qknorm_operand_t* k, const qknorm_operand_t* v, int64_t T,
           int dtype, float eps, int64_t head_dim, int64_t gstride, const qknorm_rope_t* rope,
           const qknorm_axes_t* axes, const qknorm_cache_t* cache, const int64_t* slots, void* stream) {
  RopeChecked c;
  bool noop;
  const int rc = check_rope(fn, q, k, v, T, dtype, eps, head_dim, gstride, rope, axes, cache, slots, true, &c, &noop);
  if (rc || noop) return rc;
  std::string err;
  const int mode = cache->format == QKNORM_CACHE_MXFP4   ? ROPE_APPEND_MXFP4
                   : cache->format == QKNORM_CACHE_MXFP8 ? ROPE_APPEND_MXFP8
                                                         : ROPE_APPEND_ROWS;
  if (launch_rope(mode, dtype, c.args.rot && rope->interleaved, c.plan, c.args, stream, &err))
    return fail(QKNORM_ERR_HIP, "%s: %s", fn, err.c_str());
  return ok();
}

// -------------------------------------------------------------------- gather
int gather(const char* fn, const qknorm_cache_t* cache, int64_t head_dim, const int64_t* slots, int64_t T, int dtype,
           void* k_rows, int64_t ld_k, void* v_rows, int64_t ld_v, void* stream) {
  if (!elem_size(dtype)) return fail(QKNORM_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, dtype);
  if (dtype == QKNORM_FP8_E4M3)
    return fail(QKNORM_ERR_UNSUPPORTED, "%s: FP8 rows are not supported (float32 or bf16)", fn);
  if (T < 0) return fail(QKNORM_ERR_INVALID_ARG, "%s: T = %lld < 0", fn, (long long)T);
  if (head_dim <= 0) return fail(QKNORM_ERR_INVALID_ARG, "%s: head_dim = %lld", fn, (long long)head_dim);
  if (head_dim > kRopeMaxHead)
    return fail(QKNORM_ERR_UNSUPPORTED, "%s: head_dim = %lld > %d", fn, (long long)head_dim, kRopeMaxHead);
  const int64_t esz = (int64_t)elem_size(dtype);
  int rc = check_cache(fn, cache, head_dim, esz, T > 0);
  if (rc) return rc;
  const int64_t h = cache->heads * head_dim;
  if (T > 0 && !k_rows && !v_rows) return fail(QKNORM_ERR_INVALID_ARG, "%s: k_rows or v_rows is required", fn);
  if (k_rows && (rc = check_rows(fn, "k_rows", k_rows, ld_k, h, T, esz))) return rc;
  if (v_rows && (rc = check_rows(fn, "v_rows", v_rows, ld_v, h, T, esz))) return rc;
  if (T > 0 && (!slots || !multiple(slots, 8)))
    return fail(QKNORM_ERR_INVALID_ARG, "%s: slots must be an 8-byte aligned device pointer", fn);
  if (T == 0) return ok();
  const bool codes = coded(cache);
  const Region outs[] = {Region{(uintptr_t)k_rows, ld_k, h, k_rows ? T : 0, esz},
                         Region{(uintptr_t)v_rows, ld_v, h, v_rows ? T : 0, esz}};
  const Region ins[] = {cache_region(cache, cache->k, false, head_dim, esz),
                        cache_region(cache, cache->v, false, head_dim, esz),
                        codes ? cache_region(cache, cache->k_scales, true, head_dim, esz) : Region{},
                        codes ? cache_region(cache, cache->v_scales, true, head_dim, esz) : Region{},
                        bytes_of(slots, T * 8)};
  if (may_overlap(outs[0], outs[1])) return fail(QKNORM_ERR_INVALID_ARG, "%s: k_rows overlaps v_rows", fn);
  for (const Region& out : outs)
    for (const Region& in : ins)
      if (may_overlap(out, in)) return fail(QKNORM_ERR_INVALID_ARG, "%s: the rows overlap the cache or slots", fn);

  const int64_t unit = codes ? 1 : esz;
  Aligned al;
  for (const Region& r : outs)
    if (r.T) {
      al.need((const void*)r.base, 16);
      al.need(r.ld * esz, 16);
    }
  if (!codes) {
    al.need(cache->k, 16);
    al.need(cache->v, 16);
    al.need(cache->page_stride * esz, 16);
    al.need(cache->head_stride * esz, 16);
    al.need(cache->token_stride * esz, 16);
    al.need(head_dim * esz, 16);
  }
  const int piece_bytes = al.ok ? 16 : (int)esz;
  GatherArgs a;
  std::memset(&a, 0, sizeof a);
  a.cache[0] = (const char*)cache->k;
  a.cache[1] = (const char*)cache->v;
  a.scales[0] = (const uint8_t*)cache->k_scales;
  a.scales[1] = (const uint8_t*)cache->v_scales;
  a.out[0] = (char*)k_rows;
  a.out[1] = (char*)v_rows;
  a.ld[0] = ld_k * esz;
  a.ld[1] = ld_v * esz;
  a.page_stride = cache->page_stride * unit;
  a.head_stride = cache->head_stride * unit;
  a.token_stride = cache->token_stride * unit;
  a.scale_page_stride = cache->scale_page_stride;
  a.scale_head_stride = cache->scale_head_stride;
  a.slots = slots;
  a.T = T;
  a.n_tokens_held = cache->n_pages * cache->page_size;
  a.log2_page = log2_of(cache->page_size);
  a.head_dim = (int)head_dim;
  a.pieces = (int)(head_dim * esz / (codes ? 16 : piece_bytes));
  a.items = (int)(cache->heads * a.pieces);
  a.groups = (a.items + 63) / 64 * (k_rows && v_rows ? 2 : 1);
  const int kind = cache->format == QKNORM_CACHE_ROWS    ? GATHER_ROWS
                   : cache->format == QKNORM_CACHE_MXFP4 ? GATHER_MXFP4
                                                         : GATHER_MXFP8;
  std::string err;
  if (launch_gather(kind, dtype, piece_bytes, a, stream, &err))
    return fail(QKNORM_ERR_HIP, "%s: %s", fn, err.c_str());
  return ok();
}

// Attention over MXFP4, or (wide) over rows and MXFP8.
int attend(const char* fn, bool wide, const qknorm_operand_t* q, int64_t T, int dtype, const qknorm_cache_t* cache,
           int64_t head_dim, const qknorm_batch_t* batch, float scale, int causal, int64_t window, void* workspace,
           size_t workspace_bytes, void* stream) {
  if (!q || !cache || !batch) return fail(QKNORM_ERR_INVALID_ARG, "%s: q, cache and batch are required", fn);
  if (!elem_size(dtype)) return fail(QKNORM_ERR_INVALID_ARG, "%s: unknown dtype %d", fn, dtype);
  if (dtype != QKNORM_BF16) return fail(QKNORM_ERR_UNSUPPORTED, "%s: query rows are bf16", fn);
  if (T < 0) return fail(QKNORM_ERR_INVALID_ARG, "%s: T = %lld < 0", fn, (long long)T);
  if (head_dim != 64 && head_dim != 128 && head_dim != 256)
    return fail(head_dim > 0 ? QKNORM_ERR_UNSUPPORTED : QKNORM_ERR_INVALID_ARG, "%s: head_dim = %lld (64, 128 or 256)",
                fn, (long long)head_dim);
  if (!wide && (cache->format == QKNORM_CACHE_ROWS || cache->format == QKNORM_CACHE_MXFP8))
    return fail(QKNORM_ERR_UNSUPPORTED, "%s: the cache must be MXFP4", fn);
  if (wide && cache->format == QKNORM_CACHE_MXFP4)
    return fail(QKNORM_ERR_UNSUPPORTED, "%s: the cache must be rows or MXFP8", fn);
  if (!(std::isfinite(scale) && scale > 0.0f))
    return fail(QKNORM_ERR_INVALID_ARG, "%s: scale must be finite and > 0", fn);
  if (window < 0) return fail(QKNORM_ERR_INVALID_ARG, "%s: window = %lld < 0", fn, (long long)window);
  const bool none = T == 0 || batch->B == 0;
  const bool codes = cache->format != QKNORM_CACHE_ROWS;
  const int64_t unit = codes ? 1 : 2;      // bytes of the strides' elements
  int rc = check_cache(fn, cache, head_dim, unit, !none);
  if (rc) return rc;
  if ((rc = check_width(fn, "q", q->h, head_dim))) return rc;
  const int64_t heads_q = q->h / head_dim;
  if (heads_q % cache->heads)
    return fail(QKNORM_ERR_INVALID_ARG, "%s: %lld query heads are not a multiple of %lld key heads", fn,
                (long long)heads_q, (long long)cache->heads);
  if (batch->B < 0 || batch->max_q <= 0 || batch->max_len <= 0 || batch->table_pages <= 0 ||
      batch->ld_table < batch->table_pages)
    return fail(QKNORM_ERR_INVALID_ARG, "%s: batch sizes: B >= 0, max_q, max_len and table_pages > 0, ld_table >= "
                "table_pages", fn);
  if (!batch->cu_q && T != batch->B)
    return fail(QKNORM_ERR_INVALID_ARG, "%s: without cu_q there is one query row per sequence: T = %lld, B = %lld", fn,
                (long long)T, (long long)batch->B);
  // positions a few tiles behind the last one still fit 32 bits
  if (batch->table_pages > kMaxTokens / cache->page_size)
    return fail(QKNORM_ERR_UNSUPPORTED, "%s: a table row names more than 2^30 tokens", fn);
  if (batch->ld_table > INT64_MAX / 8 / (batch->B + 1))
    return fail(QKNORM_ERR_INVALID_ARG, "%s: the block table exceeds the address range", fn);
  if ((rc = check_rows(fn, "q->x", q->x, q->ld_x, q->h, T, 2))) return rc;
  if ((rc = check_rows(fn, "q->y", q->y, q->ld_y, q->h, T, 2))) return rc;
  if (none) return ok();
  if (!multiple(q->x, 16) || !multiple(q->y, 16) || (T > 1 && (q->ld_x % 8 || q->ld_y % 8)))
    return fail(QKNORM_ERR_INVALID_ARG, "%s: query and output rows must be 16-byte aligned", fn);
  if (wide && cache->page_size < 16)
    return fail(QKNORM_ERR_UNSUPPORTED, "%s: pages of fewer than 16 tokens", fn);
  if (!codes && !(multiple(cache->k, 16) && multiple(cache->v, 16) && cache->page_stride % 8 == 0 &&
                  cache->head_stride % 8 == 0 && cache->token_stride % 8 == 0))
    return fail(QKNORM_ERR_INVALID_ARG, "%s: cache pointers and strides must be multiples of 16 bytes", fn);
  // a lane's offset among the tokens that one load takes is 32 bits
  if (cache->token_stride > (((int64_t)1 << 32) - 1024) / 16 / unit)
    return fail(QKNORM_ERR_UNSUPPORTED, "%s: cache->token_stride = %lld", fn, (long long)cache->token_stride);
  if (!batch->block_table || !batch->seq_lens)
    return fail(QKNORM_ERR_INVALID_ARG, "%s: block_table and seq_lens are required", fn);
  if (!multiple(batch->block_table, 4) || !multiple(batch->seq_lens, 4) || !multiple(batch->cu_q, 4))
    return fail(QKNORM_ERR_INVALID_ARG, "%s: batch arrays must be aligned to 4 bytes", fn);
  // The hints shape the launch; no more than there is to do.
  const int64_t capacity = batch->table_pages * cache->page_size;
  const int64_t max_q = !batch->cu_q ? 1 : batch->max_q < T ? batch->max_q : T;
  const int64_t max_len = batch->max_len < capacity ? batch->max_len : capacity;
  if (!attend_sizes_ok(T, heads_q, cache->heads, head_dim, batch->B, max_q, max_len))
    return fail(QKNORM_ERR_UNSUPPORTED, "%s: sizes beyond the kernel's limits (65536 query heads, 2^20 sequences)", fn);
  const int64_t group = heads_q / cache->heads;
  if (!attend_rows_ok(T, group))
    return fail(QKNORM_ERR_UNSUPPORTED, "%s: T = %lld query rows are too many", fn, (long long)T);
  const AttendPlan p = wide ? plan_attend_wide(codes, head_dim, cache->heads, group, batch->B, T, max_q, max_len, window)
                            : plan_attend(head_dim, cache->heads, group, batch->B, T, max_q, max_len, window);
  const int64_t block = wide && p.row_tile == 16 ? 512 : 256;
  if ((int64_t)batch->B * cache->heads * p.row_tiles > kLaunchThreads / block / p.splits)
    return fail(QKNORM_ERR_UNSUPPORTED, "%s: the launch exceeds the grid", fn);
  const size_t need = attend_workspace(p, T, heads_q);
  if (need && (!workspace || !multiple(workspace, 16) || workspace_bytes < need))
    return fail(QKNORM_ERR_INVALID_ARG, "%s: the workspace must be 16-byte aligned, at least %zu bytes", fn, need);

  const Region y{(uintptr_t)q->y, q->ld_y, q->h, T, 2};
  const Region ws = bytes_of(workspace, (int64_t)need);
  const Region ins[] = {Region{(uintptr_t)q->x, q->ld_x, q->h, T, 2},
                        cache_region(cache, cache->k, false, head_dim, unit),
                        cache_region(cache, cache->v, false, head_dim, unit),
                        codes ? cache_region(cache, cache->k_scales, true, head_dim, 1) : Region{},
                        codes ? cache_region(cache, cache->v_scales, true, head_dim, 1) : Region{},
                        bytes_of(batch->block_table, ((batch->B - 1) * batch->ld_table + batch->table_pages) * 4),
                        bytes_of(batch->seq_lens, batch->B * 4),
                        bytes_of(batch->cu_q, batch->cu_q ? (batch->B + 1) * 4 : 0)};
  for (const Region& in : ins)
    if (may_overlap(y, in) || may_overlap(ws, in))
      return fail(QKNORM_ERR_INVALID_ARG, "%s: the output or the workspace overlaps an input", fn);
  if (may_overlap(y, ws)) return fail(QKNORM_ERR_INVALID_ARG, "%s: the output overlaps the workspace", fn);

  AttendArgs a;
  std::memset(&a, 0, sizeof a);
  a.q = q->x;
  a.out = q->y;
  a.ldq = q->ld_x;
  a.ldo = q->ld_y;
  a.T = (int)T;
  a.cache[0] = (const uint8_t*)cache->k;
  a.cache[1] = (const uint8_t*)cache->v;
  a.page_stride = cache->page_stride * unit;
  a.head_stride = cache->head_stride * unit;
  a.token_stride = cache->token_stride * unit;
  if (codes) {
    a.scales[0] = (const uint8_t*)cache->k_scales;
    a.scales[1] = (const uint8_t*)cache->v_scales;
    a.scale_page_stride = cache->scale_page_stride;
    a.scale_head_stride = cache->scale_head_stride;
    a.scale_row = (int)(head_dim / 32);
  }
  a.n_pages = (uint32_t)(cache->n_pages < INT32_MAX ? cache->n_pages : INT32_MAX);
  a.log2_page = log2_of(cache->page_size);
  a.heads_k = (int)cache->heads;
  a.group = (int)(heads_q / cache->heads);
  a.table = batch->block_table;
  a.ld_table = batch->ld_table;
  a.table_tokens = (int)capacity;
  a.seq_lens = batch->seq_lens;
  a.cu_q = batch->cu_q;
  a.B = (int)batch->B;
  a.causal = causal != 0;
  a.window = window < capacity + T ? (int)window : 0;   // wider than any position: no limit
  a.scale_log2 = (float)((double)scale * 1.4426950408889634074);
  a.by_group = divisor((uint32_t)a.group);
  a.by_pairs = divisor((uint32_t)(batch->B * cache->heads));
  a.by_splits = divisor((uint32_t)p.splits);
  a.by_heads = divisor((uint32_t)cache->heads);
  a.row_tiles = p.row_tiles;
  a.splits = p.splits;
  a.chunk = p.chunk;
  a.part_o = (float*)workspace;
  a.part_ml = need ? (float*)workspace + (size_t)T * heads_q * p.splits * p.head_dim : nullptr;
  std::string err;
  if (wide ? launch_attend_wide(codes, p, a, stream, &err) : launch_attend(p, a, stream, &err))
    return fail(QKNORM_ERR_HIP, "%s: %s", fn, err.c_str());
  return ok();
}

}  // namespace

extern "C" {

int qknorm_headwise_rope(const qknorm_operand_t* q, const qknorm_operand_t* k, int64_t T, int dtype, float eps,
                         int64_t head_dim, int64_t gamma_head_stride, const qknorm_rope_t* rope, void* stream) {
  return rope_forward("qknorm_headwise_rope", q, k, T, dtype, eps, head_dim, gamma_head_stride, rope, nullptr, stream);
}

int qknorm_headwise_rope_axes(const qknorm_operand_t* q, const qknorm_operand_t* k, int64_t T, int dtype, float eps,
                              int64_t head_dim, int64_t gamma_head_stride, const qknorm_rope_t* rope,
                              const qknorm_axes_t* axes, void* stream) {
  return rope_forward("qknorm_headwise_rope_axes", q, k, T, dtype, eps, head_dim, gamma_head_stride, rope, axes, stream);
}

int qknorm_headwise_rope_backward(const qknorm_grad_operand_t* q, const qknorm_grad_operand_t* k, int64_t T,
                                  int dtype, float eps, int64_t head_dim, int64_t gamma_head_stride,
                                  const qknorm_rope_t* rope, void* workspace, size_t workspace_bytes, void* stream) {
  return rope_backward("qknorm_headwise_rope_backward", q, k, T, dtype, eps, head_dim, gamma_head_stride, rope, nullptr,
                       workspace, workspace_bytes, stream);
}

int qknorm_headwise_rope_axes_backward(const qknorm_grad_operand_t* q, const qknorm_grad_operand_t* k, int64_t T,
                                       int dtype, float eps, int64_t head_dim, int64_t gamma_head_stride,
                                       const qknorm_rope_t* rope, const qknorm_axes_t* axes, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  return rope_backward("qknorm_headwise_rope_axes_backward", q, k, T, dtype, eps, head_dim, gamma_head_stride, rope,
                       axes, workspace, workspace_bytes, stream);
}

size_t qknorm_headwise_rope_backward_workspace(int64_t hq, int64_t hk, int64_t T, int dtype, int64_t head_dim,
                                               int64_t gamma_head_stride) {
  if (T <= 0 || head_dim <= 0 || head_dim > kRopeMaxHead || hq <= 0 || hk <= 0 || hq % head_dim || hk % head_dim ||
      hq > kMaxWidth || hk > kMaxWidth || (dtype != QKNORM_F32 && dtype != QKNORM_BF16) || gamma_head_stride < 0)
    return 0;
  return grad_workspace(hq / head_dim, hk / head_dim, T, dtype, head_dim, gamma_head_stride);
}

int qknorm_paged_append(const qknorm_operand_t* q, const qknorm_operand_t* k, const qknorm_operand_t* v, int64_t T,
                        int dtype, float eps, int64_t head_dim, int64_t gamma_head_stride, const qknorm_rope_t* rope,
                        const qknorm_cache_t* cache, const int64_t* slots, void* stream) {
  return append("qknorm_paged_append", q, k, v, T, dtype, eps, head_dim, gamma_head_stride, rope, nullptr, cache, slots,
                stream);
}

int qknorm_paged_append_axes(const qknorm_operand_t* q, const qknorm_operand_t* k, const qknorm_operand_t* v, int64_t T,
                             int dtype, float eps, int64_t head_dim, int64_t gamma_head_stride,
                             const qknorm_rope_t* rope, const qknorm_axes_t* axes, const qknorm_cache_t* cache,
                             const int64_t* slots, void* stream) {
  return append("qknorm_paged_append_axes", q, k, v, T, dtype, eps, head_dim, gamma_head_stride, rope, axes, cache,
                slots, stream);
}

int qknorm_paged_gather(const qknorm_cache_t* cache, int64_t head_dim, const int64_t* slots, int64_t T, int dtype,
                        void* k_rows, int64_t ld_k, void* v_rows, int64_t ld_v, void* stream) {
  return gather("qknorm_paged_gather", cache, head_dim, slots, T, dtype, k_rows, ld_k, v_rows, ld_v, stream);
}

int qknorm_paged_attend(const qknorm_operand_t* q, int64_t T, int dtype, const qknorm_cache_t* cache,
                        int64_t head_dim, const qknorm_batch_t* batch, float scale, int causal, int64_t window,
                        void* workspace, size_t workspace_bytes, void* stream) {
  return attend("qknorm_paged_attend", false, q, T, dtype, cache, head_dim, batch, scale, causal, window, workspace,
                workspace_bytes, stream);
}

int qknorm_paged_attend_wide(const qknorm_operand_t* q, int64_t T, int dtype, const qknorm_cache_t* cache,
                             int64_t head_dim, const qknorm_batch_t* batch, float scale, int causal, int64_t window,
                             void* workspace, size_t workspace_bytes, void* stream) {
  return attend("qknorm_paged_attend_wide", true, q, T, dtype, cache, head_dim, batch, scale, causal, window,
                workspace, workspace_bytes, stream);
}

size_t qknorm_paged_attend_workspace(int64_t T, int64_t heads_q, int64_t heads_k, int64_t head_dim, int64_t B,
                                     int64_t max_q, int64_t max_len) {
  if (!attend_sizes_ok(T, heads_q, heads_k, head_dim, B, max_q, max_len) || T == 0 || B == 0 ||
      !attend_rows_ok(T, heads_q / heads_k))
    return 0;
  return attend_workspace(plan_attend(head_dim, heads_k, heads_q / heads_k, B, T, max_q < T ? max_q : T, max_len, 0),
                          T, heads_q);
}

size_t qknorm_paged_attend_wide_workspace(int64_t T, int64_t heads_q, int64_t heads_k, int64_t head_dim, int64_t B,
                                          int64_t max_q, int64_t max_len) {
  if (!attend_sizes_ok(T, heads_q, heads_k, head_dim, B, max_q, max_len) || T == 0 || B == 0 ||
      !attend_rows_ok(T, heads_q / heads_k))
    return 0;
  return attend_workspace(
      plan_attend_wide(true, head_dim, heads_k, heads_q / heads_k, B, T, max_q < T ? max_q : T, max_len, 0), T, heads_q);
}

}  // extern "C"

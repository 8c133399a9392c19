"""Binding of the operators around headwise QK-Norm: the norm with the
position rotation in the same pass, its gradients, appending to a paged key /
value cache and attention over the 4-bit cache (argument marshalling only, as
``binding.py``; the C names are kept).

The calls run on torch's current stream of the tensors' device, whichever
device is current, or on ``stream``. What a call allocates itself (outputs or
a workspace that were not passed) belongs to the stream it runs on.
"""

import ctypes
import math

from .binding import (CACHE_MXFP4, CACHE_ROWS, Batch, Cache, GradOperand, Operand, PreparedCall, Rope, _check,
                      _dtype_code, _gamma_dtype, _rows, _same_device, _stream, _tokens, _torch_mod, load_library)


def rope_table(n_positions, rot_dim, base=10000.0, inv_freq=None, device="cuda"):
    """The float32 table [n_positions, rot_dim] that the rotating calls read: row p
    holds cos(p f_i), then sin(p f_i), with f_i = base^(-2i / rot_dim) or
    ``inv_freq`` [rot_dim / 2]. Angles are formed in float64, so far positions
    keep their accuracy."""
    torch = _torch_mod()
    if rot_dim <= 0 or rot_dim % 2:
        raise ValueError(f"rot_dim must be even and positive, got {rot_dim}")
    if inv_freq is None:
        i = torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device)
        inv_freq = float(base) ** (-i / rot_dim)
    else:
        inv_freq = torch.as_tensor(inv_freq, device=device).to(torch.float64)
        if tuple(inv_freq.shape) != (rot_dim // 2,):
            raise ValueError(f"inv_freq must have shape ({rot_dim // 2},)")
    angle = torch.arange(n_positions, dtype=torch.float64, device=device)[:, None] * inv_freq[None, :]
    return torch.cat((angle.cos(), angle.sin()), 1).to(torch.float32)


class _OperatorCall(PreparedCall):
    """A PreparedCall that also makes its tensors' device the current one for the launch."""

    def __call__(self, stream=None):
        torch = _torch_mod()
        if torch.cuda.current_device() != self._device:
            with torch.cuda.device(self._device):
                return super().__call__(stream)
        return super().__call__(stream)


def _run(fn, args, t, stream):
    """Enqueues fn(*args, stream) on the stream, with t's device current."""
    torch = _torch_mod()
    s = _stream(t, stream)
    dev = t.get_device()
    if torch.cuda.current_device() == dev:
        _check(fn(*args, s))
    else:   # the default stream is the current device's own
        with torch.cuda.device(dev):
            _check(fn(*args, s))


def _empty(shape, dtype, t, stream):
    """New memory on t's device that belongs to the stream the call runs on."""
    torch = _torch_mod()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=t.device)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=t.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=t.device)


def _vector(t, n, dtype, ref, name):
    if t.dtype != dtype or t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} must be a contiguous {dtype} vector of {n}")
    _same_device(t, ref, name)
    return t.data_ptr()


def _rope(cos_sin, positions, interleaved, T, ref):
    if cos_sin is None:
        return None
    torch = _torch_mod()
    if cos_sin.dtype != torch.float32 or cos_sin.dim() != 2 or (cos_sin.shape[1] > 1 and cos_sin.stride(1) != 1):
        raise ValueError("cos_sin must be a float32 table [n_positions, rot_dim] with contiguous rows")
    _same_device(cos_sin, ref, "cos_sin")
    n, rot = cos_sin.shape
    return Rope(cos_sin.data_ptr(), cos_sin.stride(0) if n > 1 else max(cos_sin.stride(0), rot), n,
                _vector(positions, T, torch.int64, ref, "positions"), rot, int(bool(interleaved)))


def _gamma(gamma, x, head_dim, gstride, name):
    if gamma is None:
        return None
    need = (x.shape[1] // head_dim - 1) * gstride + head_dim if head_dim > 0 and gstride >= 0 else 0
    if gamma.dim() != 1 or gamma.shape[0] < need or (gamma.shape[0] > 1 and gamma.stride(0) != 1) \
            or gamma.dtype != _gamma_dtype(x):
        raise ValueError(f"gamma for {name} must be contiguous, dtype {_gamma_dtype(x)}, >= {need} elements")
    _same_device(gamma, x, "gamma for " + name)
    return gamma.data_ptr()


def _like(y, x, name):
    """Row stride of rows y that go with rows x."""
    if y.shape != x.shape or y.dtype != x.dtype:
        raise ValueError(f"{name} must have shape {tuple(x.shape)} and dtype {x.dtype}")
    _same_device(y, x, name)
    return _rows(y, name)


def _side(x, y, gamma, head_dim, gstride, name):
    o = Operand()
    o.ld_x = _rows(x, name)
    o.x = x.data_ptr()
    o.h = x.shape[1]
    if y is not None:
        o.ld_y = _like(y, x, "output for " + name)
        o.y = y.data_ptr()
    o.gamma = _gamma(gamma, x, head_dim, gstride, name)
    return o


def _ref(p):
    return None if p is None else ctypes.byref(p)


# ---------------------------------------------------------------- norm and rotation
def _headwise_rope(q, k, gamma_q, gamma_k, eps, head_dim, cos_sin, positions, interleaved, gamma_head_stride, out_q,
                   out_k):
    T = _tokens(q, k)
    if gamma_q is None or gamma_k is None:
        raise ValueError("gamma_q and gamma_k are required")
    out_q = q if out_q is None else out_q
    out_k = k if out_k is None else out_k
    head_dim, gs = int(head_dim), int(gamma_head_stride)
    oq = _side(q, out_q, gamma_q, head_dim, gs, "q")
    ok = _side(k, out_k, gamma_k, head_dim, gs, "k")
    rope = _rope(cos_sin, positions, interleaved, T, q)
    args = (_ref(oq), _ref(ok), T, _dtype_code(q), float(eps), head_dim, gs, _ref(rope))
    return args, (oq, ok, rope), (out_q, out_k)


def qknorm_headwise_rope(q, k, gamma_q, gamma_k, eps, head_dim, cos_sin, positions, interleaved=False,
                         gamma_head_stride=0, out_q=None, out_k=None, stream=None):
    """Headwise QK-Norm of q [T, hq] and k [T, hk], then the rotation of every head's
    first ``cos_sin.shape[1]`` columns by its token's angles, in one pass.

    cos_sin: float32 [n_positions, rot_dim], cos then sin (``rope_table``), or None for no
    rotation; positions: int64 [T]. interleaved pairs columns (2i, 2i + 1) instead of
    (i, i + rot_dim / 2). Writes ``out_q``/``out_k`` (default: in place) and returns them."""
    args, _, out = _headwise_rope(q, k, gamma_q, gamma_k, eps, head_dim, cos_sin, positions, interleaved,
                                  gamma_head_stride, out_q, out_k)
    _run(load_library().qknorm_headwise_rope, args, q, stream)
    return out


def prepare_headwise_rope(q, k, gamma_q, gamma_k, eps, head_dim, cos_sin, positions, interleaved=False,
                          gamma_head_stride=0, out_q=None, out_k=None):
    """qknorm_headwise_rope with its arguments checked and marshalled once (PreparedCall)."""
    args, held, out = _headwise_rope(q, k, gamma_q, gamma_k, eps, head_dim, cos_sin, positions, interleaved,
                                     gamma_head_stride, out_q, out_k)
    return _OperatorCall(load_library().qknorm_headwise_rope, args,
                         (q, k, gamma_q, gamma_k, cos_sin, positions, out, held), q.get_device(), out)


# ------------------------------------------------------------------------ gradients
def _headwise_rope_backward(dy_q, dy_k, q, k, gamma_q, gamma_k, eps, head_dim, cos_sin, positions, interleaved,
                            gamma_head_stride, dx_q, dx_k, dgamma_q, dgamma_k, need_dgamma, workspace, stream):
    torch = _torch_mod()
    lib = load_library()
    T = _tokens(q, k)
    if gamma_q is None or gamma_k is None:
        raise ValueError("gamma_q and gamma_k are required")
    head_dim, gs = int(head_dim), int(gamma_head_stride)
    sides, outs = [], []
    for x, dy, dx, gamma, dgamma, name in ((q, dy_q, dx_q, gamma_q, dgamma_q, "q"),
                                           (k, dy_k, dx_k, gamma_k, dgamma_k, "k")):
        o = GradOperand()
        o.ld_x, o.x, o.h = _rows(x, name), x.data_ptr(), x.shape[1]
        o.ld_dy, o.dy = _like(dy, x, "dy_" + name), dy.data_ptr()
        if dx is None:
            dx = _empty(tuple(x.shape), x.dtype, x, stream)
        o.ld_dx, o.dx = _like(dx, x, "dx_" + name), dx.data_ptr()
        o.gamma = _gamma(gamma, x, head_dim, gs, name)
        if dgamma is None and need_dgamma:
            # columns that no head has (a stride past head_dim) and the case of no tokens stay 0
            whole = T > 0 and gs <= head_dim and head_dim > 0 \
                and gamma.shape[0] == (x.shape[1] // head_dim - 1) * gs + head_dim
            dgamma = _empty(tuple(gamma.shape), torch.float32, x, stream)
            if not whole:
                _zero(dgamma, stream)
        if dgamma is not None:
            if dgamma.dtype != torch.float32 or dgamma.shape != gamma.shape \
                    or (dgamma.shape[0] > 1 and dgamma.stride(0) != 1):
                raise ValueError(f"dgamma_{name} must be contiguous float32 {tuple(gamma.shape)}")
            _same_device(dgamma, x, "dgamma_" + name)
            o.dgamma = dgamma.data_ptr()
        sides.append(o)
        outs.append((dx, dgamma))
    code = _dtype_code(q)
    need = lib.qknorm_headwise_rope_backward_workspace(q.shape[1], k.shape[1], T, code, head_dim, gs)
    if workspace is None and (outs[0][1] is not None or outs[1][1] is not None):
        workspace = _empty((need,), torch.uint8, q, stream)
    ws, ws_bytes = _workspace(workspace, q)
    rope = _rope(cos_sin, positions, interleaved, T, q)
    args = (_ref(sides[0]), _ref(sides[1]), T, code, float(eps), head_dim, gs, _ref(rope), ws, ws_bytes)
    return args, (sides, rope, workspace), (outs[0][0], outs[1][0], outs[0][1], outs[1][1])


def _zero(t, stream):
    torch = _torch_mod()
    if stream is None:
        t.zero_()
        return
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=t.device)
    with torch.cuda.stream(stream):
        t.zero_()


def _workspace(workspace, ref):
    if workspace is None:
        return None, 0
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    _same_device(workspace, ref, "workspace")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size()


def qknorm_headwise_rope_backward(dy_q, dy_k, q, k, gamma_q, gamma_k, eps, head_dim, cos_sin, positions,
                                  interleaved=False, gamma_head_stride=0, dx_q=None, dx_k=None, dgamma_q=None,
                                  dgamma_k=None, need_dgamma=True, workspace=None, stream=None):
    """Gradients of ``qknorm_headwise_rope`` (with cos_sin None, of ``qknorm_headwise``) for
    the output gradients dy_q [T, hq] and dy_k [T, hk] at the inputs q and k.

    Returns (dx_q, dx_k, dgamma_q, dgamma_k): dx in the row type, dgamma float32 in gamma's
    layout (None without need_dgamma, where none was passed). Outputs that are not passed
    are allocated. workspace: uint8, at least ``qknorm_headwise_rope_backward_workspace``
    bytes; allocated if None."""
    args, _, out = _headwise_rope_backward(dy_q, dy_k, q, k, gamma_q, gamma_k, eps, head_dim, cos_sin, positions,
                                           interleaved, gamma_head_stride, dx_q, dx_k, dgamma_q, dgamma_k,
                                           need_dgamma, workspace, stream)
    _run(load_library().qknorm_headwise_rope_backward, args, q, stream)
    return out


def prepare_headwise_rope_backward(dy_q, dy_k, q, k, gamma_q, gamma_k, eps, head_dim, cos_sin, positions,
                                   interleaved=False, gamma_head_stride=0, dx_q=None, dx_k=None, dgamma_q=None,
                                   dgamma_k=None, need_dgamma=True, workspace=None):
    """qknorm_headwise_rope_backward with its arguments checked and marshalled once
    (PreparedCall). It keeps its workspace: calls of one object must not run at the same
    time on two streams."""
    args, held, out = _headwise_rope_backward(dy_q, dy_k, q, k, gamma_q, gamma_k, eps, head_dim, cos_sin, positions,
                                              interleaved, gamma_head_stride, dx_q, dx_k, dgamma_q, dgamma_k,
                                              need_dgamma, workspace, None)
    return _OperatorCall(load_library().qknorm_headwise_rope_backward, args,
                         (dy_q, dy_k, q, k, gamma_q, gamma_k, cos_sin, positions, out, held), q.get_device(), out)


# ---------------------------------------------------------------------- paged cache
def _cache(k_cache, v_cache, k_scales, v_scales, head_dim, ref, row_dtype):
    """Cache of [pages, heads, page_size, head_dim] tensors (any strides with contiguous
    heads), or of uint8 codes [.., head_dim / 2] with uint8 scales [.., head_dim / 32]."""
    torch = _torch_mod()
    four = k_scales is not None or v_scales is not None
    if four and (k_scales is None or v_scales is None):
        raise ValueError("k_scales and v_scales go together")
    last = head_dim // 2 if four else head_dim
    dtype = torch.uint8 if four else row_dtype
    for t, name in ((k_cache, "k_cache"), (v_cache, "v_cache")):
        if t.dim() != 4 or t.shape[3] != last or t.dtype != dtype or (last > 1 and t.stride(3) != 1):
            raise ValueError(f"{name} must be {dtype} [pages, heads, page_size, {last}] with a contiguous last axis")
        _same_device(t, ref, name)
    if k_cache.shape != v_cache.shape or k_cache.stride() != v_cache.stride():
        raise ValueError("k_cache and v_cache must have the same shape and strides")
    n, heads, ps, _ = k_cache.shape

    def strides(t, inner):
        # an axis of length one may carry any stride: what it would hold is a valid one
        s = list(t.stride())
        if t.shape[2] == 1:
            s[2] = inner
        if t.shape[1] == 1:
            s[1] = max(s[1], s[2] * t.shape[2])
        if t.shape[0] == 1:
            s[0] = max(s[0], s[1] * t.shape[1], s[2] * t.shape[2])
        return s

    s = strides(k_cache, last)
    c = Cache(CACHE_MXFP4 if four else CACHE_ROWS, k_cache.data_ptr(), v_cache.data_ptr(), None, None, s[0], s[1],
              s[2], 0, 0, n, ps, heads)
    if four:
        blocks = head_dim // 32
        for t, name in ((k_scales, "k_scales"), (v_scales, "v_scales")):
            if tuple(t.shape) != (n, heads, ps, blocks) or t.dtype != torch.uint8 \
                    or (blocks > 1 and t.stride(3) != 1) or (ps > 1 and t.stride(2) != blocks):
                raise ValueError(f"{name} must be uint8 [{n}, {heads}, {ps}, {blocks}], a head's tokens packed")
            _same_device(t, ref, name)
        if k_scales.stride() != v_scales.stride():
            raise ValueError("k_scales and v_scales must have the same strides")
        ss = strides(k_scales, blocks)
        c.k_scales, c.v_scales = k_scales.data_ptr(), v_scales.data_ptr()
        c.scale_page_stride, c.scale_head_stride = ss[0], ss[1]
    return c


def _paged_append(q, k, v, gamma_q, gamma_k, eps, head_dim, cos_sin, positions, k_cache, v_cache, slots, k_scales,
                  v_scales, interleaved, gamma_head_stride, out_q, out_k, out_v):
    torch = _torch_mod()
    T = _tokens(k, v)
    head_dim, gs = int(head_dim), int(gamma_head_stride)
    oq = None
    if q is not None:
        _tokens(q, k)
        out_q = q if out_q is None else out_q
        oq = _side(q, out_q, gamma_q, head_dim, gs, "q")
    ok = _side(k, out_k, gamma_k, head_dim, gs, "k")
    ov = _side(v, out_v, None, head_dim, gs, "v")
    cache = _cache(k_cache, v_cache, k_scales, v_scales, head_dim, k, k.dtype)
    rope = _rope(cos_sin, positions, interleaved, T, k)
    args = (_ref(oq), _ref(ok), _ref(ov), T, _dtype_code(k), float(eps), head_dim, gs, _ref(rope), _ref(cache),
            _vector(slots, T, torch.int64, k, "slots"))
    return args, (oq, ok, ov, cache, rope), out_q


def qknorm_paged_append(q, k, v, gamma_q, gamma_k, eps, head_dim, cos_sin, positions, k_cache, v_cache, slots,
                        k_scales=None, v_scales=None, interleaved=False, gamma_head_stride=0, out_q=None, out_k=None,
                        out_v=None, stream=None):
    """A step's keys and values into a paged cache and its queries made ready, in one pass:
    q [T, hq] normalized and rotated into ``out_q`` (default: in place; q may be None), k
    normalized and rotated into k_cache, v into v_cache.

    gamma_q / gamma_k None: that side is rotated only. k_cache, v_cache: the row type
    [pages, heads, page_size, head_dim], or with k_scales and v_scales (uint8 [.., head_dim / 32])
    MXFP4 codes, uint8 [.., head_dim / 2]. slots: int64 [T], page * page_size + place; a token
    with a negative slot is passed over (nothing of its row is written). out_k / out_v, if
    given, receive as rows what the cache now holds. Returns out_q."""
    args, _, out = _paged_append(q, k, v, gamma_q, gamma_k, eps, head_dim, cos_sin, positions, k_cache, v_cache,
                                 slots, k_scales, v_scales, interleaved, gamma_head_stride, out_q, out_k, out_v)
    _run(load_library().qknorm_paged_append, args, k, stream)
    return out


def prepare_paged_append(q, k, v, gamma_q, gamma_k, eps, head_dim, cos_sin, positions, k_cache, v_cache, slots,
                         k_scales=None, v_scales=None, interleaved=False, gamma_head_stride=0, out_q=None,
                         out_k=None, out_v=None):
    """qknorm_paged_append with its arguments checked and marshalled once (PreparedCall)."""
    args, held, out = _paged_append(q, k, v, gamma_q, gamma_k, eps, head_dim, cos_sin, positions, k_cache, v_cache,
                                    slots, k_scales, v_scales, interleaved, gamma_head_stride, out_q, out_k, out_v)
    return _OperatorCall(load_library().qknorm_paged_append, args,
                         (q, k, v, gamma_q, gamma_k, cos_sin, positions, k_cache, v_cache, slots, k_scales, v_scales,
                          out_q, out_k, out_v, held), k.get_device(), out)


def _paged_attend(q, k_cache, v_cache, k_scales, v_scales, block_table, seq_lens, head_dim, cu_q, scale, causal,
                  window, max_q, max_len, out, workspace, stream):
    torch = _torch_mod()
    lib = load_library()
    if k_scales is None or v_scales is None:
        raise ValueError("k_scales and v_scales are required: the cache is MXFP4")
    head_dim = int(head_dim)
    oq = Operand()
    oq.ld_x = _rows(q, "q")
    T, h = q.shape
    oq.x, oq.h = q.data_ptr(), h
    if out is None:
        out = _empty((T, h), q.dtype, q, stream)
    oq.ld_y, oq.y = _like(out, q, "out"), out.data_ptr()
    cache = _cache(k_cache, v_cache, k_scales, v_scales, head_dim, q, q.dtype)
    if block_table.dim() != 2 or block_table.dtype != torch.int32 \
            or (block_table.shape[1] > 1 and block_table.stride(1) != 1):
        raise ValueError("block_table must be int32 [B, pages] with contiguous rows")
    _same_device(block_table, q, "block_table")
    B, pages = block_table.shape
    ld = block_table.stride(0) if B > 1 else max(block_table.stride(0), pages)
    lens = _vector(seq_lens, B, torch.int32, q, "seq_lens")
    cu = None if cu_q is None else _vector(cu_q, B + 1, torch.int32, q, "cu_q")
    capacity = pages * cache.page_size
    max_q = (1 if cu is None else max(T, 1)) if max_q is None else int(max_q)
    max_len = capacity if max_len is None else min(int(max_len), capacity)
    if head_dim > 0 and scale is None:
        scale = 1.0 / math.sqrt(head_dim)
    batch = Batch(block_table.data_ptr(), ld, pages, lens, cu, B, max_q, max_len)
    if workspace is None and head_dim > 0:
        need = lib.qknorm_paged_attend_workspace(T, h // head_dim, cache.heads, head_dim, B,
                                                 1 if cu is None else max_q, max_len)
        if need:
            workspace = _empty((need,), torch.uint8, q, stream)
    ws, ws_bytes = _workspace(workspace, q)
    args = (_ref(oq), T, _dtype_code(q), _ref(cache), head_dim, _ref(batch), float(scale or 0.0), int(bool(causal)),
            int(window or 0), ws, ws_bytes)
    return args, (oq, cache, batch, workspace), out


def qknorm_paged_attend(q, k_cache, v_cache, k_scales, v_scales, block_table, seq_lens, head_dim, cu_q=None,
                        scale=None, causal=True, window=0, max_q=None, max_len=None, out=None, workspace=None,
                        stream=None):
    """Attention of bf16 query rows q [T, heads * head_dim] over a paged MXFP4 cache
    (``qknorm_paged_append``'s layout); head_dim 64, 128 or 256.

    block_table: int32 [B, pages]; seq_lens: int32 [B], this call's tokens included; cu_q:
    int32 [B + 1] first query row of each sequence, None for one query row per sequence.
    causal, window: what a query sees (window 0: no limit). scale: default 1/sqrt(head_dim).
    max_q, max_len: the caller's bounds on query rows and cached tokens of a sequence (they
    shape the launch; default: what the shapes allow). workspace: uint8, at least
    ``qknorm_paged_attend_workspace`` bytes; allocated if None. Returns ``out`` (allocated if
    None); rows outside every sequence are not written."""
    args, _, out = _paged_attend(q, k_cache, v_cache, k_scales, v_scales, block_table, seq_lens, head_dim, cu_q,
                                 scale, causal, window, max_q, max_len, out, workspace, stream)
    _run(load_library().qknorm_paged_attend, args, q, stream)
    return out


def prepare_paged_attend(q, k_cache, v_cache, k_scales, v_scales, block_table, seq_lens, head_dim, cu_q=None,
                         scale=None, causal=True, window=0, max_q=None, max_len=None, out=None, workspace=None):
    """qknorm_paged_attend with its arguments checked and marshalled once (PreparedCall): for
    decode loops, whose seq_lens and block_table change in place between calls. It keeps its
    workspace: calls of one object must not run at the same time on two streams."""
    args, held, out = _paged_attend(q, k_cache, v_cache, k_scales, v_scales, block_table, seq_lens, head_dim, cu_q,
                                    scale, causal, window, max_q, max_len, out, workspace, None)
    return _OperatorCall(load_library().qknorm_paged_attend, args,
                         (q, k_cache, v_cache, k_scales, v_scales, block_table, seq_lens, cu_q, out, held),
                         q.get_device(), out)

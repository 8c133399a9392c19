"""Binding of the operators around headwise QK-Norm: the norm with the
position rotation in the same pass, its gradients, appending to a paged key /
value cache and attention over the 4-bit cache (argument marshalling only, in
the C++ module ``_qknorm_torch``; the C names are kept).

The calls run on torch's current stream of the tensors' device, whichever
device is current, or on ``stream``. What a call allocates itself (outputs or
a workspace that were not passed) belongs to the stream it runs on. What a
prepared call allocates belongs to the stream that is current at its
preparation; launches on other streams are recorded on it, so that dropping the
call hands none of it out again while a launch still uses it. A prepared call
that a graph has captured has to be kept as long as the graph is replayed.
"""

import importlib
import os

import torch

from .binding import PreparedCall, QKNormError, _check, load_library

_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_module = None


def _native():
    """The marshalling module, loaded with libqknorm.so on first use."""
    global _module
    if _module is None:
        load_library()
        if not os.path.exists(os.path.join(os.path.dirname(os.path.abspath(__file__)), "_qknorm_torch.so")):
            raise QKNormError(-1, "_qknorm_torch.so is not built; run __graft_entry__.build()")
        _module = importlib.import_module("._qknorm_torch", __package__)
    return _module


def rope_table(n_positions, rot_dim, base=10000.0, inv_freq=None, device="cuda"):
    """The float32 table [n_positions, rot_dim] that the rotating calls read: row p
    holds cos(p f_i), then sin(p f_i), with f_i = base^(-2i / rot_dim) or
    ``inv_freq`` [rot_dim / 2]. Angles are formed in float64, so far positions
    keep their accuracy."""
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
    """A PreparedCall whose marshalled arguments the native module holds (with
    their tensors), and that makes its tensors' device the current one. `own` is
    what was allocated for it, on the stream that is current now."""

    def __init__(self, call, device, result, own=()):
        super().__init__(None, (), (), device, result)
        self._call = call
        self._own = own
        self._known = {_handle(device, None)}    # streams that the allocator knows to use `own`

    def __call__(self, stream=None):
        s = _handle(self._device, stream)
        if self._own and s not in self._known:
            on = _torch_stream(s if stream is None else stream, torch.device("cuda", self._device))
            for t in self._own:
                t.record_stream(on)
            self._known.add(s)
        _on(self._device, s, lambda s: _native().launch(self._call, s))
        return self._result


def _handle(dev, stream):
    """The stream handle a call runs on: `stream`'s, or that of the device's current stream."""
    if stream is not None:
        return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
    return _raw_stream(dev) if _raw_stream is not None else torch.cuda.current_stream(dev).cuda_stream


def _on(dev, s, enqueue):
    """enqueue(stream handle) with `dev` current: the default stream is the current device's own."""
    if _current_device() == dev:
        rc = enqueue(s)
    else:
        with torch.cuda.device(dev):
            rc = enqueue(s)
    if rc:
        _check(rc)


def _run(name, args, rows, stream):
    """The native call on rows' device. (A tensor that is not on a GPU is refused there.)"""
    fn = getattr(_module or _native(), name)
    dev = rows.get_device() if isinstance(rows, torch.Tensor) else -1
    if stream is None and dev >= 0 and _raw_stream is not None and _current_device() == dev:
        rc = fn(*args, _raw_stream(dev), False)
        if rc:
            _check(rc)
    elif dev < 0:
        fn(*args, 0, True)      # raises: the rows are not on a GPU
        raise ValueError("the rows must be device tensors")
    else:
        _on(dev, _handle(dev, stream), lambda s: fn(*args, s, False))


def _prepared(name, args, rows, result, own=()):
    call = getattr(_native(), name)(*args, 0, True)
    return _OperatorCall(call, rows.get_device(), result, tuple(t for t in own if t is not None))


def _torch_stream(stream, device):
    """torch's stream for a stream object or handle. Handle 0 is the device's default stream
    (ExternalStream would take it for no handle, and make a stream of its own)."""
    if hasattr(stream, "cuda_stream"):
        return stream
    handle = int(stream)
    return torch.cuda.ExternalStream(handle, device=device) if handle else torch.cuda.default_stream(device)


def _current(rows):
    """The current stream of rows' device (None: not on a GPU, which the native module refuses)."""
    return torch.cuda.current_stream(rows.device) if rows.is_cuda else None


def _at(stream, device):
    """Context in which new memory belongs to the stream a call runs on."""
    return torch.cuda.stream(None if stream is None else _torch_stream(stream, device))     # None: no change


# ---------------------------------------------------------------- norm and rotation
def qknorm_headwise_rope(q, k, gamma_q, gamma_k, eps, head_dim, cos_sin, positions, interleaved=False,
                         gamma_head_stride=0, out_q=None, out_k=None, stream=None):
    """Headwise QK-Norm of q [T, hq] and k [T, hk], then the rotation of every head's
    first ``cos_sin.shape[1]`` columns by its token's angles, in one pass.

    cos_sin: float32 [n_positions, rot_dim], cos then sin (``rope_table``), or None for no
    rotation; positions: int64 [T]. interleaved pairs columns (2i, 2i + 1) instead of
    (i, i + rot_dim / 2). Writes ``out_q``/``out_k`` (default: in place) and returns them."""
    _run("rope", (q, k, gamma_q, gamma_k, eps, head_dim, cos_sin, positions, interleaved, gamma_head_stride, out_q,
                  out_k), q, stream)
    return (q if out_q is None else out_q), (k if out_k is None else out_k)


def prepare_headwise_rope(q, k, gamma_q, gamma_k, eps, head_dim, cos_sin, positions, interleaved=False,
                          gamma_head_stride=0, out_q=None, out_k=None):
    """qknorm_headwise_rope with its arguments checked and marshalled once (PreparedCall)."""
    return _prepared("rope", (q, k, gamma_q, gamma_k, eps, head_dim, cos_sin, positions, interleaved,
                              gamma_head_stride, out_q, out_k), q,
                     (q if out_q is None else out_q, k if out_k is None else out_k))


# ------------------------------------------------------------------------ gradients
def _new_gradient(gamma, x, head_dim, stride):
    """dgamma for gamma: elements that no head has, and all of them for no tokens, are 0."""
    heads = x.shape[1] // head_dim if head_dim > 0 else 0
    if x.shape[0] and stride <= head_dim and gamma.shape[0] == (heads - 1) * stride + head_dim:
        return torch.empty(gamma.shape, dtype=torch.float32, device=x.device)
    return torch.zeros(gamma.shape, dtype=torch.float32, device=x.device)


def _gradient_outputs(q, k, gamma_q, gamma_k, head_dim, stride, dx_q, dx_k, dgamma_q, dgamma_k, need_dgamma,
                      workspace, on):
    """The outputs and the workspace that were not passed, in memory of the stream `on`."""
    if on is not None or dx_q is None or dx_k is None or (need_dgamma and (dgamma_q is None or dgamma_k is None)):
        if gamma_q is None or gamma_k is None:
            raise ValueError("gamma_q and gamma_k are required")
        with _at(on, q.device):
            if dx_q is None:
                dx_q = torch.empty(q.shape, dtype=q.dtype, device=q.device)
            if dx_k is None:
                dx_k = torch.empty(k.shape, dtype=k.dtype, device=k.device)
            if need_dgamma:
                dgamma_q = _new_gradient(gamma_q, q, head_dim, stride) if dgamma_q is None else dgamma_q
                dgamma_k = _new_gradient(gamma_k, k, head_dim, stride) if dgamma_k is None else dgamma_k
            if workspace is None and on is not None and not (dgamma_q is None and dgamma_k is None):
                code = {torch.float32: 0, torch.bfloat16: 1}.get(q.dtype, 2)
                need = load_library().qknorm_headwise_rope_backward_workspace(
                    q.shape[1], k.shape[1], q.shape[0], code, int(head_dim), int(stride))
                workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    return dx_q, dx_k, dgamma_q, dgamma_k, workspace


def qknorm_headwise_rope_backward(dy_q, dy_k, q, k, gamma_q, gamma_k, eps, head_dim, cos_sin, positions,
                                  interleaved=False, gamma_head_stride=0, dx_q=None, dx_k=None, dgamma_q=None,
                                  dgamma_k=None, need_dgamma=True, workspace=None, stream=None):
    """Gradients of ``qknorm_headwise_rope`` (with cos_sin None, of ``qknorm_headwise``) for
    the output gradients dy_q [T, hq] and dy_k [T, hk] at the inputs q and k.

    Returns (dx_q, dx_k, dgamma_q, dgamma_k): dx in the row type, dgamma float32 in gamma's
    layout (None without need_dgamma, where none was passed). Outputs that are not passed
    are allocated. workspace: uint8, at least ``qknorm_headwise_rope_backward_workspace``
    bytes; allocated if None."""
    dx_q, dx_k, dgamma_q, dgamma_k, workspace = _gradient_outputs(
        q, k, gamma_q, gamma_k, head_dim, gamma_head_stride, dx_q, dx_k, dgamma_q, dgamma_k, need_dgamma, workspace,
        stream)
    _run("rope_backward", (dy_q, dy_k, q, k, gamma_q, gamma_k, eps, head_dim, cos_sin, positions, interleaved,
                           gamma_head_stride, dx_q, dx_k, dgamma_q, dgamma_k, workspace), q, stream)
    return dx_q, dx_k, dgamma_q, dgamma_k


def prepare_headwise_rope_backward(dy_q, dy_k, q, k, gamma_q, gamma_k, eps, head_dim, cos_sin, positions,
                                   interleaved=False, gamma_head_stride=0, dx_q=None, dx_k=None, dgamma_q=None,
                                   dgamma_k=None, need_dgamma=True, workspace=None):
    """qknorm_headwise_rope_backward with its arguments checked and marshalled once
    (PreparedCall). It keeps its workspace: calls of one object must not run at the same
    time on two streams."""
    given = (dx_q, dx_k, dgamma_q, dgamma_k, workspace)
    made = _gradient_outputs(q, k, gamma_q, gamma_k, head_dim, gamma_head_stride, *given[:4], need_dgamma, workspace,
                             _current(q))
    return _prepared("rope_backward", (dy_q, dy_k, q, k, gamma_q, gamma_k, eps, head_dim, cos_sin, positions,
                                       interleaved, gamma_head_stride, *made), q, made[:4],
                     (m for m, g in zip(made, given) if g is None))


# ---------------------------------------------------------------------- paged cache
def qknorm_paged_append(q, k, v, gamma_q, gamma_k, eps, head_dim, cos_sin, positions, k_cache, v_cache, slots,
                        k_scales=None, v_scales=None, interleaved=False, gamma_head_stride=0, out_q=None, out_k=None,
                        out_v=None, stream=None):
    """A step's keys and values into a paged cache and its queries made ready, in one pass:
    q [T, hq] normalized and rotated into ``out_q`` (default: in place; q may be None), k
    normalized and rotated into k_cache, v into v_cache.

    gamma_q / gamma_k None: that side is rotated only. k_cache, v_cache: the row type
    [pages, heads, page_size, head_dim], or with k_scales and v_scales (uint8 [.., head_dim / 32])
    MXFP4 codes, uint8 [.., head_dim / 2]. slots: int64 [T], page * page_size + place; a token
    with a negative slot is passed over (nothing of its row is written), and no two may have
    the same. out_k / out_v, if given, receive as rows what the cache now holds. Returns out_q."""
    _run("append", (q, k, v, gamma_q, gamma_k, eps, head_dim, cos_sin, positions, k_cache, v_cache, slots, k_scales,
                    v_scales, interleaved, gamma_head_stride, out_q, out_k, out_v), k, stream)
    return q if out_q is None else out_q


def prepare_paged_append(q, k, v, gamma_q, gamma_k, eps, head_dim, cos_sin, positions, k_cache, v_cache, slots,
                         k_scales=None, v_scales=None, interleaved=False, gamma_head_stride=0, out_q=None,
                         out_k=None, out_v=None):
    """qknorm_paged_append with its arguments checked and marshalled once (PreparedCall)."""
    return _prepared("append", (q, k, v, gamma_q, gamma_k, eps, head_dim, cos_sin, positions, k_cache, v_cache, slots,
                                k_scales, v_scales, interleaved, gamma_head_stride, out_q, out_k, out_v), k,
                     q if out_q is None else out_q)


def _attend_memory(q, k_cache, block_table, head_dim, cu_q, max_q, max_len, out, workspace, stream):
    """The output and the workspace that were not passed, in memory of `stream`."""
    if out is None or (stream is not None and workspace is None):
        with _at(stream, q.device):
            if out is None:
                out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
            if stream is not None and workspace is None and head_dim > 0 and k_cache.dim() == 4:
                capacity = block_table.shape[1] * k_cache.shape[2]
                need = load_library().qknorm_paged_attend_workspace(
                    q.shape[0], q.shape[1] // head_dim, k_cache.shape[1], head_dim, block_table.shape[0],
                    1 if cu_q is None else max(q.shape[0], 1) if max_q is None else max_q,
                    capacity if max_len is None else min(max_len, capacity))
                workspace = torch.empty(need, dtype=torch.uint8, device=q.device) if need else None
    return out, workspace


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
    out, workspace = _attend_memory(q, k_cache, block_table, head_dim, cu_q, max_q, max_len, out, workspace, stream)
    _run("attend", (q, k_cache, v_cache, k_scales, v_scales, block_table, seq_lens, head_dim, cu_q, scale, causal,
                    window, max_q, max_len, out, workspace), q, stream)
    return out


def prepare_paged_attend(q, k_cache, v_cache, k_scales, v_scales, block_table, seq_lens, head_dim, cu_q=None,
                         scale=None, causal=True, window=0, max_q=None, max_len=None, out=None, workspace=None):
    """qknorm_paged_attend with its arguments checked and marshalled once (PreparedCall): for
    decode loops, whose seq_lens and block_table change in place between calls. It keeps its
    workspace: calls of one object must not run at the same time on two streams."""
    given = (out, workspace)
    made = _attend_memory(q, k_cache, block_table, head_dim, cu_q, max_q, max_len, out, workspace,
                          _current(q))
    return _prepared("attend", (q, k_cache, v_cache, k_scales, v_scales, block_table, seq_lens, head_dim, cu_q, scale,
                                causal, window, max_q, max_len, *made), q, made[0],
                     (m for m, g in zip(made, given) if g is None))

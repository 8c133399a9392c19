"""Shared by the tests of the operators around headwise QK-Norm: seeded host
inputs, device copies, and the tolerances, each derived from the arithmetic
before it was first used.

u = 2^-24 is half a step of float32. With n-term float32 sums of positive
squares the RMS factor is off by at most about (chain + 6 butterfly steps +
4) u / 2; chains here are at most 32 terms, so z = x gamma r is within 32 u.
"""

import numpy as np
import torch

from gpu_helpers import DEV, np_to_torch, torch_to_np
from oracle.bf16 import bf16_bits_to_f64, f64_to_bf16_bits
from oracle.fp8 import f64_to_fp8_bits, fp8_bits_to_f64

U = 2.0 ** -24
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "fp8": 2.0 ** -4}     # half a step, relative
LOWEST = {"f32": 0.0, "bf16": 2.0 ** -134, "fp8": 2.0 ** -10}       # half a subnormal step
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}


def rng(seed):
    return np.random.Generator(np.random.PCG64(seed))


def to_type(x, dtype):
    """float64 -> host storage of the row type."""
    if dtype == "f32":
        return x.astype(np.float32)
    if dtype == "bf16":
        return f64_to_bf16_bits(x.astype(np.float32).astype(np.float64))
    return f64_to_fp8_bits(np.clip(x, -448, 448))


def values(h):
    """Host storage -> float64."""
    if h.dtype == np.uint16:
        return bf16_bits_to_f64(h)
    if h.dtype == np.uint8:
        return fp8_bits_to_f64(h)
    return h.astype(np.float64)


def dev(h):
    if h.dtype in (np.int32, np.int64):
        return torch.from_numpy(np.ascontiguousarray(h)).to(DEV)
    return np_to_torch(h).to(DEV)


def codes_to_dev(h):
    return torch.from_numpy(np.ascontiguousarray(h)).to(DEV)


def host_values(t):
    return values(torch_to_np(t))


def table(n, rot, base=10000.0):
    f = base ** (-np.arange(0, rot, 2) / rot)
    a = np.arange(n)[:, None] * f[None, :]
    return np.concatenate((np.cos(a), np.sin(a)), 1).astype(np.float32)


def same_bits(a, b):
    view = {1: torch.uint8, 2: torch.int16, 4: torch.int32, 8: torch.int64}[a.element_size()]
    return torch.equal(a.contiguous().view(view), b.contiguous().view(view))


def close(got, want, bound, what):
    """|got - want| <= bound elementwise, NaN and infinities in the same places."""
    assert got.shape == want.shape, (got.shape, want.shape)
    assert np.array_equal(np.isnan(got), np.isnan(want)), f"{what}: NaN in other places"
    fin = np.isfinite(want)
    inf = ~fin & ~np.isnan(want)
    assert np.array_equal(got[inf], want[inf]), f"{what}: infinities differ"
    over = np.abs(got[fin] - want[fin]) - (bound[fin] if np.ndim(bound) else bound)
    assert over.size == 0 or over.max() <= 0, \
        f"{what}: {int((over > 0).sum())} of {over.size} values beyond the bound, the worst by {over.max():.3g}"


def rope_bound(z, cos, sin, interleaved, dtype):
    """Bound on |kernel - oracle| of the rotated rows: z [T, heads, d] the unrotated values.
    A rotated value is two products of values within 32 u, one more rounding each and one of
    their sum: 36 u of |a c| + |b s|; then the rounding to the row type."""
    from oracle.operators import rotate
    mag = np.abs(z) if cos is None else rotate(np.abs(z), np.abs(cos), -np.abs(sin), interleaved)
    if cos is not None:     # both members with plus signs
        from oracle.operators import pair_columns
        first, second = pair_columns(2 * cos.shape[1], interleaved)
        a, b = np.abs(z[..., first]), np.abs(z[..., second])
        mag = np.abs(z).copy()
        mag[..., first] = a * np.abs(cos)[:, None] + b * np.abs(sin)[:, None]
        mag[..., second] = b * np.abs(cos)[:, None] + a * np.abs(sin)[:, None]
    half = HALF[dtype] if dtype != "f32" else 0.0
    return mag * (36 * U + half) * 1.01 + LOWEST[dtype]

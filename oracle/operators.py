"""Float64 oracle of the operators around headwise QK-Norm: the rotation, the
gradients, MXFP4 blocks, the paged append and attention over a paged cache.
Test infrastructure only, as the rest of this package. Everything takes and
returns plain float64 arrays (or integer codes); roundings to row types are
the caller's.
"""

import numpy as np

# E2M1 (OCP Microscaling Formats v1.0): magnitudes by code, the sign is bit 3.
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def pair_columns(rot, interleaved):
    """Columns of the first and second member of every rotated pair."""
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def rotate(x, cos, sin, interleaved, back=False):
    """x [T, heads, d]; cos, sin [T, rot/2]: each pair turned by its angle (back: by its
    negative)."""
    y = np.array(x, dtype=np.float64)
    first, second = pair_columns(2 * cos.shape[1], interleaved)
    s = -sin if back else sin
    a, b = x[..., first], x[..., second]
    y[..., first] = a * cos[:, None] - b * s[:, None]
    y[..., second] = b * cos[:, None] + a * s[:, None]
    return y


def angles(table, positions, rot):
    """cos and sin [T, rot/2] of the table's rows; NaN for positions outside it."""
    n = table.shape[0]
    inside = (positions >= 0) & (positions < n)
    rows = np.where(inside[:, None], table.astype(np.float64)[np.where(inside, positions, 0)], np.nan)
    return rows[:, :rot // 2], rows[:, rot // 2:rot]


def gamma_rows(gamma, heads, head_dim, stride):
    """gamma as [heads, head_dim]."""
    at = np.arange(heads)[:, None] * stride + np.arange(head_dim)[None, :]
    return gamma.astype(np.float64)[at]


def norm_rope(x, gamma, eps, head_dim, stride, cos, sin, interleaved):
    """x [T, heads * head_dim] -> [T, heads, head_dim]; gamma None: no norm; cos None: no rotation."""
    T, h = x.shape
    z = x.astype(np.float64).reshape(T, h // head_dim, head_dim)
    if gamma is not None:
        ms = (z * z).sum(-1, keepdims=True) / head_dim
        z = z * gamma_rows(gamma, h // head_dim, head_dim, stride) / np.sqrt(ms + np.float64(np.float32(eps)))
    return z if cos is None else rotate(z, cos, sin, interleaved)


def norm_rope_backward(x, dy, gamma, eps, head_dim, stride, cos, sin, interleaved):
    """(dx [T, heads, d], dgamma in gamma's layout, and both again with every term taken by its
    magnitude, the two products of a turned gradient among them: for tolerances)."""
    T, h = x.shape
    heads = h // head_dim
    z = x.astype(np.float64).reshape(T, heads, head_dim)
    g = dy.astype(np.float64).reshape(T, heads, head_dim)
    g_mag = np.abs(g)
    if cos is not None:
        first, second = pair_columns(2 * cos.shape[1], interleaved)
        a, b, c, s = g_mag[..., first], g_mag[..., second], np.abs(cos)[:, None], np.abs(sin)[:, None]
        g_mag = g_mag.copy()
        g_mag[..., first], g_mag[..., second] = a * c + b * s, b * c + a * s
        g = rotate(g, cos, sin, interleaved, back=True)
    r = 1.0 / np.sqrt((z * z).sum(-1, keepdims=True) / head_dim + np.float64(np.float32(eps)))
    gam = gamma_rows(gamma, heads, head_dim, stride)
    xr, gg = z * r, g * gam
    mean = (gg * xr).mean(-1, keepdims=True)
    dx = r * (gg - xr * mean)
    gg_mag = g_mag * np.abs(gam)
    dx_mag = r * (gg_mag + np.abs(xr) * (gg_mag * np.abs(xr)).mean(-1, keepdims=True))
    terms, terms_mag = g * xr, g_mag * np.abs(xr)
    dgamma, dgamma_mag = np.zeros(gamma.shape), np.zeros(gamma.shape)
    for i in range(heads):
        sl = slice(i * stride, i * stride + head_dim)
        dgamma[sl] += terms[:, i].sum(0)
        dgamma_mag[sl] += terms_mag[:, i].sum(0)
    return dx, dgamma, dx_mag, dgamma_mag


def mxfp4_quantize(x):
    """x [..., d] (d a multiple of 32) -> (codes uint8 [..., d/2], scale bytes uint8 [..., d/32],
    values float64 [..., d]). Scale 2^E with E = floor(log2(largest magnitude)) - 2 held to
    [-100, 125]; the nearest E2M1 value, ties to the even code, at most 6; a block with an
    infinity or NaN: codes 0, scale byte 255, values NaN."""
    x = np.asarray(x, np.float64)
    b = x.reshape(*x.shape[:-1], -1, 32)
    ok = np.isfinite(b).all(-1)
    safe = np.where(ok[..., None], b, 0.0)
    amax = np.abs(safe).max(-1)
    _, e = np.frexp(amax)                       # amax = m 2^e, m in [1/2, 1)
    E = np.where(amax > 0, np.clip(e - 3, -100, 125), -100)
    a = np.ldexp(np.abs(safe), -E[..., None])
    gap = np.abs(a[..., None] - E2M1)           # distance to every value
    gap = np.where(np.arange(8) % 2 == 1, np.nextafter(gap, np.inf), gap)   # even codes win ties
    code = gap.argmin(-1)
    value = np.ldexp(E2M1[code], E[..., None]) * np.where(np.signbit(safe), -1.0, 1.0)
    code = code + 8 * np.signbit(safe)
    code = code.reshape(x.shape).astype(np.uint8)
    packed = code[..., 0::2] | (code[..., 1::2] << 4)
    scale = np.where(ok, E + 127, 255).astype(np.uint8)
    return packed, scale, np.where(ok[..., None], value, np.nan).reshape(x.shape)


def mxfp4_values(codes, scales):
    """float64 values of codes [..., d/2] with scale bytes [..., d/32]; bytes above 252: NaN."""
    code = np.stack((codes & 15, codes >> 4), -1).reshape(*codes.shape[:-1], 2 * codes.shape[-1])
    x = E2M1[code & 7] * np.where(code & 8, -1.0, 1.0)
    s = np.where(scales <= 252, np.ldexp(1.0, scales.astype(np.int64) - 127), np.nan)
    return x * np.repeat(s, 32, axis=-1)


def attend(q, K, V, n_q, scale, causal, window):
    """One sequence: q [n_q, heads_q, d], K, V [len, heads_k, d] (all cached tokens) ->
    (out [n_q, heads_q, d], sum of p |v| [same], rows that see something [n_q])."""
    n, heads_k = K.shape[0], K.shape[1]
    heads_q, d = q.shape[1], q.shape[2]
    out, mag = np.zeros((n_q, heads_q, d)), np.zeros((n_q, heads_q, d))
    some = np.zeros(n_q, bool)
    for i in range(n_q):
        pos = n - n_q + i
        hi = 0 if pos < 0 else (pos + 1 if causal else n)
        lo = max(0, pos - window + 1) if window else 0
        if hi <= lo:
            continue
        some[i] = True
        for h in range(heads_q):
            kh = h // (heads_q // heads_k)
            s = K[lo:hi, kh] @ q[i, h] * scale
            with np.errstate(invalid="ignore"):
                p = np.exp(s - s.max())
                p = p / p.sum()
                out[i, h] = p @ V[lo:hi, kh]
                mag[i, h] = p @ np.abs(V[lo:hi, kh])
    return out, mag, some

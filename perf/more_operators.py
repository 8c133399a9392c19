"""More operators around headwise QK-Norm, as cases to measure: the rotation by
positions of several axes (time, height, width) with the norm, its gradients,
appending to a cache that is quantised as it is written (MXFP8: E4M3 codes, one
E8M0 scale per 32 channels of a head), reading a cache back as rows, and
attention of new tokens over a paged cache of bf16 rows or MXFP8.

With ``own`` false every case runs in elementary torch operations (float32,
float64 where codes are decided); with ``own`` true it makes the framework's
calls on the same inputs.
"""

import math
import random

import torch

own = False

EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "fp8": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f32": 4, "fp8": 1}
LOWEST_EXPONENT = -100
# elements to a byte of codes, largest scale exponent, log2 of the largest code's leading bit
MX = {"mxfp4": (2, 125, 2), "mxfp8": (1, 119, 8)}
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases
def _case(name, op, **kw):
    c = {"name": name, "op": op, "dtype": "bf16", "head_dim": 128}
    c.update(kw)
    return c


def listed():
    return [
        # one image through a vision encoder: two axes, multi-head, heads of 80
        _case("axes_image", "axes", T=1024, heads_q=16, heads_k=16, head_dim=80, rot=80, n_axes=2, spread=False,
              interleaved=False, per_head=False, n_pos=64),
        # a video prompt of a grouped-query model: time, height and width in sections of the angles
        _case("axes_prompt", "axes", T=8192, heads_q=40, heads_k=8, rot=128, n_axes=3, spread=False,
              interleaved=False, per_head=False, n_pos=8192),
        # gradients of a training batch of it
        _case("axes_grad_batch", "grad", T=8192, heads_q=40, heads_k=8, rot=128, n_axes=3, spread=False,
              interleaved=False, per_head=False, n_pos=8192),
        # gradients on one tensor-parallel slice, float32, axes dealt to the angles in turn, full-width gamma
        _case("axes_grad_slice", "grad", T=1000, heads_q=10, heads_k=2, rot=128, n_axes=3, spread=True,
              interleaved=False, per_head=True, n_pos=1024, dtype="f32"),
        # a decode step of 64 sequences into the 8-bit cache
        _case("append_tokens", "append", T=64, heads_q=40, heads_k=8, rot=128, n_axes=0, spread=False,
              interleaved=False, norm=True, n_pos=32768, page=16, cache="mxfp8"),
        # a video prompt into the 8-bit cache
        _case("append_prompt", "append", T=8192, heads_q=40, heads_k=8, rot=128, n_axes=3, spread=False,
              interleaved=False, norm=True, n_pos=8192, page=64, cache="mxfp8"),
        # a shared prefix read back from the 8-bit cache as bf16 rows
        _case("gather_prefix", "gather", T=16384, heads_q=8, heads_k=8, page=64, cache="mxfp8"),
        # a few hundred tokens read back from the 4-bit cache, in float32, to be written elsewhere
        _case("gather_tokens", "gather", T=333, heads_q=8, heads_k=8, page=16, cache="mxfp4", dtype="f32"),
        # a decode batch of uneven lengths on a bf16 cache, one of them empty
        _case("attend_batch", "attend", B=64, q=1, len=8192, heads_q=40, heads_k=8, page=64, window=0, causal=True,
              empty=True, cache="rows"),
        # one sequence with a long 8-bit cache: the axis has to be split
        _case("attend_long", "attend", B=1, q=1, len=65536, heads_q=40, heads_k=8, page=16, window=0, causal=True,
              cache="mxfp8"),
        # a short step of a multi-head model, a few drafted tokens each: latency
        _case("attend_short", "attend", B=4, q=5, len=333, heads_q=32, heads_k=32, page=16, window=0, causal=True,
              cache="mxfp8"),
        # prompts read in chunks behind what the cache already holds
        _case("attend_chunk", "attend", B=4, q=1024, len=8192, heads_q=40, heads_k=8, page=32, window=0,
              causal=True, cache="rows"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("axes", "grad", "append", "gather", "attend", "attend"))
    heads_k = rng.choice((1, 2, 3, 4, 8))
    group = rng.choice((1, 2, 4, 5, 7, 8))
    c = {"op": op, "heads_q": heads_k * group, "heads_k": heads_k}
    if op == "attend":
        c["head_dim"] = rng.choice((64, 128, 128, 256))
        c["dtype"] = "bf16"
        c["cache"] = rng.choice(("rows", "mxfp8"))
        c["page"] = rng.choice((16, 32, 64, 128))
        c["causal"] = rng.random() < 0.85
        c["window"] = rng.choice((0, 0, _log(rng, 16, 4096)))
        if rng.random() < 0.5:       # decode, or a few tokens a step
            c["q"] = rng.choice((1, 1, 1, 2, 5))
            c["B"] = _log(rng, 1, 96)
            c["len"] = max(c["q"], _log(rng, 1, 8192))
        else:                        # prompts and chunks
            c["B"] = rng.choice((1, 2, 3))
            c["q"] = _log(rng, 8, 1024)
            c["len"] = c["q"] + _log(rng, 1, 4096) - 1
        c["empty"] = c["B"] > 2 and rng.random() < 0.3
        return c
    c["T"] = _log(rng, 1, 8192)
    if op == "gather":
        c["cache"] = rng.choice(("mxfp8", "mxfp8", "mxfp4", "rows"))
        c["dtype"] = rng.choice(("bf16", "bf16", "f32"))
        c["head_dim"] = rng.choice((64, 96, 128, 128, 256))
        c["page"] = rng.choice((16, 32, 64, 128))
        return c
    c["dtype"] = rng.choice(("bf16", "bf16", "f32", "fp8") if op == "axes" else ("bf16", "bf16", "f32"))
    c["head_dim"] = rng.choice((64, 80, 96, 128, 128, 256))
    c["n_axes"] = rng.choice((2, 3, 3))
    if op == "append":
        c["cache"] = rng.choice(("mxfp8", "mxfp8", "mxfp8", "mxfp4", "rows"))
        if c["cache"] == "mxfp8":
            c["n_axes"] = rng.choice((0, 2, 3))
        c["head_dim"] = rng.choice((64, 96, 128, 128, 256))
        c["page"] = rng.choice((16, 32, 64, 128))
        c["norm"] = rng.random() < 0.7
    else:
        c["per_head"] = rng.random() < 0.3
    c["spread"] = rng.random() < 0.3
    c["interleaved"] = rng.random() < 0.4
    c["rot"] = rng.choice((c["head_dim"], c["head_dim"], c["head_dim"] // 2))
    c["n_pos"] = _log(rng, 256, 65536)
    while c["T"] * c["heads_q"] * c["head_dim"] > 8192 * 5120:
        c["T"] //= 2
    return c


# ------------------------------------------------------------------ sizes
def _lengths(c):
    """Cache lengths and query counts of the sequences: set by the case, not by the seed."""
    r = random.Random(c["B"] * 6007 + c["len"])
    lens, nqs = [], []
    for b in range(c["B"]):
        nq = c["q"] if b == 0 or c["q"] == 1 else r.randint(max(1, c["q"] // 2), c["q"])
        n = c["len"] if b == 0 else max(nq, r.randint((c["len"] + 1) // 2, c["len"]))
        lens.append(n)
        nqs.append(nq)
    if c.get("empty"):
        lens[-1] = 0
    return lens, nqs


def _visible(c):
    """(cached tokens any query of a sequence sees, summed; query-token pairs, summed)."""
    tokens = pairs = 0
    for n, nq in zip(*_lengths(c)):
        first = n
        for i in range(nq):
            pos = n - nq + i
            hi = min(n, pos + 1) if c["causal"] else n
            lo = max(0, pos - c["window"] + 1) if c["window"] else 0
            if hi > lo:
                pairs += hi - lo
                first = min(first, lo)
        tokens += n - first
    return tokens, pairs


def _held(c, elements):
    """Bytes of that many elements in the case's cache."""
    if c["cache"] == "rows":
        return elements * BYTES[c["dtype"]]
    return elements // MX[c["cache"]][0] + elements // 32


def work(c):
    e = BYTES[c["dtype"]]
    d, hq, hk = c["head_dim"], c["heads_q"], c["heads_k"]
    if c["op"] == "attend":
        tokens, pairs = _visible(c)
        rows = sum(_lengths(c)[1])
        return {"bytes": _held(c, tokens * hk * 2 * d) + 2 * rows * hq * d * e, "flops": 4 * pairs * hq * d}
    T, w, kv = c["T"], (hq + hk) * d, 2 * c["T"] * hk * d
    if c["op"] == "gather":
        return {"bytes": _held(c, kv) + kv * e + 8 * T, "flops": kv}
    table = min(T, c["n_pos"]) * c["rot"] * 4 + 8 * T * max(1, c["n_axes"])
    gamma = (hq + hk if c.get("per_head") else 2) * d * max(e, 2)
    if c["op"] == "axes":
        return {"bytes": 2 * T * w * e + table + gamma, "flops": 9 * T * w}
    if c["op"] == "grad":
        return {"bytes": 3 * T * w * e + table + gamma + gamma // e * 4, "flops": 18 * T * w}
    rows = kv * e if c["cache"] != "rows" else 0     # the values that the cache now holds, as rows
    return {"bytes": 2 * T * hq * d * e + kv * e + _held(c, kv) + rows + table + 8 * T,
            "flops": 9 * T * (w + hk * d)}


# ------------------------------------------------------------------ inputs
def _axis_of(c):
    """The axis of every angle, as bytes: time takes a quarter of three axes' angles, height and width share the
    rest (16, 24 and 24 of 64); two axes share evenly. spread: dealt in turn while they last."""
    n = c["rot"] // 2
    if c["n_axes"] == 2:
        left = [(n + 1) // 2, n // 2]
    else:
        left = [n // 4, (n - n // 4 + 1) // 2, (n - n // 4) // 2]
    if not c["spread"]:
        return bytes(a for a, m in enumerate(left) for _ in range(m))
    out, a = [], 0
    while len(out) < n:
        if left[a]:
            left[a] -= 1
            out.append(a)
        a = (a + 1) % len(left)
    return bytes(out)


def _table(n_pos, rot, dev):
    """cos and sin of every position's angles, formed in float64: [n_pos, rot], cos first."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=dev) / rot)
    a = torch.arange(n_pos, dtype=torch.float64, device=dev)[:, None] * f[None, :]
    return torch.cat((a.cos(), a.sin()), 1).float()


def _grid_positions(c, g):
    """[n_axes, T]: text, where the axes agree, and between it images and clips, whose tokens walk through a
    grid's columns, rows and frames. Decode: every token of a sequence of its own."""
    T, A, n, dev = c["T"], c["n_axes"], c["n_pos"], g.device
    if T <= 256 and c["op"] == "append":
        return torch.randint(0, n, (A, T), generator=g, device=dev)
    wide = int(torch.randint(4, 33, (1,), generator=g, device=dev))
    i = torch.arange(T, device=dev)
    block, at = i // 512, i % 512
    col, row = at % wide, at // wide
    walk = torch.stack((row // wide, row % wide, col)[3 - A:])
    text = (block % 4 == 0) & (A == 3)
    return (torch.where(text, i, block * 64 + walk) % n).contiguous()


def _normal(g, shape, dtype, scale=1.0, mean=0.0):
    x = torch.randn(shape, generator=g, device=g.device, dtype=torch.float32) * scale + mean
    if dtype == torch.float8_e4m3fn:
        x = x.clamp(-448.0, 448.0)
    return x.to(dtype)


def _fill_cache(c, g, pages, s):
    """K and V of random tokens in the case's format."""
    shape = (pages, c["heads_k"], c["page"], c["head_dim"])
    for n in ("k", "v"):
        s[n + "_scales"] = None
        if c["cache"] == "rows":
            s[n + "_cache"] = torch.empty(shape, dtype=DTYPES[c["dtype"]], device=g.device)
        else:
            s[n + "_cache"] = torch.empty((*shape[:3], shape[3] // MX[c["cache"]][0]), dtype=torch.uint8,
                                          device=g.device)
            s[n + "_scales"] = torch.empty((*shape[:3], shape[3] // 32), dtype=torch.uint8, device=g.device)
        for p in range(0, pages, 512):
            x = _normal(g, (min(512, pages - p), *shape[1:]), torch.float32)
            if c["cache"] == "rows":
                s[n + "_cache"][p:p + 512] = x.to(DTYPES[c["dtype"]])
            else:
                s[n + "_cache"][p:p + 512], s[n + "_scales"][p:p + 512] = _quantize(x, c["cache"])[:2]


def prepare(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    dt = DTYPES[c["dtype"]]
    d, hq, hk = c["head_dim"], c["heads_q"], c["heads_k"]
    s = {"case": c}
    if c["op"] == "attend":
        lens, nqs = _lengths(c)
        ps, B = c["page"], c["B"]
        per = max(1, -(-max(lens) // ps))
        need = [-(-n // ps) for n in lens]
        pages = max(1, sum(need))
        order = torch.randperm(pages, generator=g, device=dev).int()
        table = torch.zeros((B, per), dtype=torch.int32, device=dev)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        _fill_cache(c, g, pages, s)
        rows = sum(nqs)
        # queries after their norm; the gamma of a trained model sharpens the scores
        s["q"] = _normal(g, (rows, hq * d), dt, 1.7)
        s["out"] = torch.zeros((rows, hq * d), dtype=dt, device=dev)
        s["block_table"] = table
        s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
        cu = [0]
        for n in nqs:
            cu.append(cu[-1] + n)
        s["cu_q"] = torch.tensor(cu, dtype=torch.int32, device=dev) if c["q"] > 1 else None
        s["max_q"], s["max_len"] = max(nqs), max(lens)
        return s
    T = c["T"]
    if c["op"] in ("append", "gather"):
        ps = c["page"]
        pages = -(-T // ps) + 3
        s["slots"] = torch.randperm(pages * ps, generator=g, device=dev)[:T] if T <= 256 else (
            torch.randperm(pages, generator=g, device=dev)[:, None] * ps
            + torch.arange(ps, device=dev)[None, :]).reshape(-1)[:T].contiguous()
        if T > 8:
            s["slots"][T - 3:] = -1                  # a padded batch: rows that hold no token
    if c["op"] == "gather":
        _fill_cache(c, g, pages, s)
        for n in ("k", "v"):
            s["out_" + n] = torch.zeros((T, hk * d), dtype=dt, device=dev)
        return s
    gdt = torch.bfloat16 if c["dtype"] == "fp8" else dt
    s["cos_sin"] = _table(c["n_pos"], c["rot"], dev)
    if c["n_axes"]:
        s["axes"] = _axis_of(c)
        s["positions"] = _grid_positions(c, g)
    elif T <= 256:    # decode
        s["positions"] = torch.randint(0, c["n_pos"], (T,), generator=g, device=dev)
    else:             # prompts one after the other
        s["positions"] = torch.arange(T, device=dev) % c["n_pos"]
    s["gamma_head_stride"] = d if c.get("per_head") else 0
    s["gamma_q"] = _normal(g, (hq * d if c.get("per_head") else d,), gdt, 0.1, 1.0)
    s["gamma_k"] = _normal(g, (hk * d if c.get("per_head") else d,), gdt, 0.1, 1.0)
    qkv = _normal(g, (T, (hq + 2 * hk) * d), dt)     # rows as the projection writes them
    s["q"], s["k"], s["v"] = qkv[:, :hq * d], qkv[:, hq * d:(hq + hk) * d], qkv[:, (hq + hk) * d:]
    if c["op"] == "append":
        if not c["norm"]:
            s["gamma_q"] = s["gamma_k"] = None
        s["out_q"] = torch.zeros((T, hq * d), dtype=dt, device=dev)
        if c["cache"] == "rows":
            for n in ("k_cache", "v_cache"):
                s[n] = _normal(g, (pages, hk, ps, d), dt)
            s["k_scales"] = s["v_scales"] = s["out_k"] = s["out_v"] = None
        else:
            for n in ("k", "v"):
                s[n + "_cache"] = torch.zeros((pages, hk, ps, d // MX[c["cache"]][0]), dtype=torch.uint8, device=dev)
                s[n + "_scales"] = torch.full((pages, hk, ps, d // 32), 127, dtype=torch.uint8, device=dev)
                s["out_" + n] = torch.zeros((T, hk * d), dtype=dt, device=dev)
        return s
    if c["op"] == "axes":
        s["out_q"] = torch.empty((T, hq * d), dtype=dt, device=dev)
        s["out_k"] = torch.empty((T, hk * d), dtype=dt, device=dev)
    else:
        s["dy_q"], s["dy_k"] = _normal(g, (T, hq * d), dt), _normal(g, (T, hk * d), dt)
        for n in ("q", "k"):
            s["dx_" + n] = torch.empty_like(s["dy_" + n])
            s["dgamma_" + n] = torch.empty(s["gamma_" + n].shape, dtype=torch.float32, device=dev)
    return s


# ------------------------------------------------------------------ the plain forms
def _quantize(x, cache):
    """x [..., d] -> codes (MXFP4: two to a byte, the even channel low), scale bytes [..., d / 32] and the values
    they stand for. Nearest code, ties to the even one."""
    _, top, lead = MX[cache]
    b = x.reshape(*x.shape[:-1], -1, 32)
    amax = b.abs().amax(-1)
    # floor(log2(amax)) from the exponent: amax = m 2^e with m in [1/2, 1)
    e = (torch.frexp(amax)[1] - 1 - lead).clamp(LOWEST_EXPONENT, top)
    e = torch.where(amax == 0, torch.full_like(e, LOWEST_EXPONENT), e)
    a = torch.ldexp(b.abs(), -e.unsqueeze(-1))
    # a code's step: one (E2M1) or three (E4M3) bits behind its leading one, never below the subnormals'
    bits, low = (1, 0) if cache == "mxfp4" else (3, -6)
    step = (torch.frexp(a)[1] - 1).clamp(min=low) - bits
    a = torch.ldexp(torch.round(torch.ldexp(a, -step)), step).clamp(max=6.0 if cache == "mxfp4" else 448.0)
    value = torch.copysign(torch.ldexp(a, e.unsqueeze(-1)), b).reshape(x.shape)
    a = torch.copysign(a, b).reshape(x.shape).float()
    scale = (e + 127).to(torch.uint8)
    if cache == "mxfp8":
        return a.to(torch.float8_e4m3fn).view(torch.uint8), scale, value
    code = torch.zeros_like(a, dtype=torch.uint8)
    for v in E2M1[1:]:
        code += (a.abs() >= v).to(torch.uint8)
    code |= torch.signbit(a).to(torch.uint8) << 3
    return code[..., 0::2] | (code[..., 1::2] << 4), scale, value


def _dequantize(cache, codes, scales):
    """The float32 values of a cache's entries (rows: as they are)."""
    if cache == "rows":
        return codes.float()
    if cache == "mxfp8":
        x = codes.view(torch.float8_e4m3fn).float()
    else:
        grid = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float32, device=codes.device)
        x = torch.stack((grid[(codes & 15).long()], grid[(codes >> 4).long()]), -1).flatten(-2)
    return torch.ldexp(x, (scales.int() - 127).repeat_interleave(32, -1))


def _angles(s, wide):
    """cos and sin [T, 1, rot / 2]: every angle at the position of its axis."""
    c = s["case"]
    half = c["rot"] // 2
    pos = s["positions"]
    if not c["n_axes"]:
        cs = s["cos_sin"].to(wide)[pos]
        return cs[:, None, :half], cs[:, None, half:]
    axis = torch.tensor(list(s["axes"]), device=pos.device)
    at = pos[axis].t()                                             # [T, rot / 2]
    i = torch.arange(half, device=pos.device)
    cs = s["cos_sin"].to(wide)
    return cs[at, i][:, None], cs[at, half + i][:, None]


def _pairs(x, rot, interleaved):
    """The two members of every rotated pair."""
    return (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])


def _join(a, b, rest, interleaved):
    head = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((head, rest), -1)


def _norm_rope(s, x, gamma, wide):
    """[T, heads * d] rows -> [T, heads, d] normalized per head (gamma None: not) and rotated."""
    c = s["case"]
    d, rot = c["head_dim"], c["rot"]
    x = x.to(wide).reshape(x.shape[0], -1, d)
    if gamma is not None:
        gamma = gamma.to(wide).reshape(1, -1, d)
        eps = torch.tensor(EPS, dtype=torch.float32, device=x.device).to(wide)
        x = x * gamma * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps)
    cos, sin = _angles(s, wide)
    a, b = _pairs(x, rot, c["interleaved"])
    return _join(a * cos - b * sin, b * cos + a * sin, x[..., rot:], c["interleaved"])


def _round(x, dt):
    return (x.clamp(-448.0, 448.0) if dt == torch.float8_e4m3fn else x).to(dt)


def _plain_grad(s, x, dy, gamma):
    c = s["case"]
    d, rot = c["head_dim"], c["rot"]
    x32 = x.float().reshape(x.shape[0], -1, d)
    g = dy.float().reshape(x.shape[0], -1, d)
    cos, sin = _angles(s, torch.float32)
    a, b = _pairs(g, rot, c["interleaved"])          # the rotation's transpose
    g = _join(a * cos + b * sin, b * cos - a * sin, g[..., rot:], c["interleaved"])
    r = torch.rsqrt((x32 * x32).mean(-1, keepdim=True) + EPS)
    xr = x32 * r
    gg = g * gamma.float().reshape(1, -1, d)
    dx = r * (gg - xr * (gg * xr).mean(-1, keepdim=True))
    dgamma = (g * xr).to(torch.float64).sum((0, 1) if gamma.numel() == d else 0)   # a long sum
    return dx.reshape(x.shape).to(x.dtype), dgamma.reshape(-1).float()


def _plain_append(s):
    c = s["case"]
    d, ps, T = c["head_dim"], c["page"], c["T"]
    coded = c["cache"] != "rows"
    keep = s["slots"] >= 0
    q = _norm_rope(s, s["q"], s["gamma_q"], torch.float32).reshape(T, -1).to(s["q"].dtype)
    s["out_q"].copy_(torch.where(keep[:, None], q, s["out_q"]))
    # codes are decided next to borders: in 64 bits
    k = _norm_rope(s, s["k"], s["gamma_k"], torch.float64 if coded else torch.float32)
    v = s["v"].reshape(T, -1, d)
    # a token without a slot writes over the first token's entry what the first token writes
    row = torch.where(keep, torch.arange(T, device=keep.device), torch.zeros_like(s["slots"]))
    slot = s["slots"][row]
    page, off = slot // ps, slot % ps
    if not coded:
        s["k_cache"][page, :, off] = k.to(s["k"].dtype)[row]
        s["v_cache"][page, :, off] = v[row]
        return {"q": s["out_q"], "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    for n, x in (("k", k), ("v", v.float())):
        codes, scales, values = _quantize(x, c["cache"])
        s[n + "_cache"][page, :, off] = codes[row]
        s[n + "_scales"][page, :, off] = scales[row]
        out = s["out_" + n]
        out.copy_(torch.where(keep[:, None], values.reshape(T, -1).to(out.dtype), out))
    return {"q": s["out_q"], "k_values": s["out_k"], "v_values": s["out_v"]}


def _plain_gather(s):
    c = s["case"]
    keep = s["slots"] >= 0
    at = torch.where(keep, s["slots"], torch.zeros_like(s["slots"]))
    page, off = at // c["page"], at % c["page"]
    for n in ("k", "v"):
        scales = s[n + "_scales"]
        x = _dequantize(c["cache"], s[n + "_cache"][page, :, off], None if scales is None else scales[page, :, off])
        out = s["out_" + n]
        out.copy_(torch.where(keep[:, None], x.reshape(c["T"], -1).to(out.dtype), out))
    return {"k": s["out_k"], "v": s["out_v"]}


def _plain_attend(s):
    c = s["case"]
    d, hq, hk, B = c["head_dim"], c["heads_q"], c["heads_k"], c["B"]
    G, dev = hq // hk, s["q"].device
    L, nq, rows = max(1, s["max_len"]), s["max_q"], s["q"].shape[0]
    at = s["block_table"].long()[:, :-(-L // c["page"])]           # [B, pages]

    def cached(n):                                                 # -> [B * hk, tokens, d]
        scales = s[n + "_scales"]
        x = _dequantize(c["cache"], s[n + "_cache"][at], None if scales is None else scales[at])
        return x.transpose(1, 2).reshape(B * hk, -1, d)

    lens = s["seq_lens"].long()[:, None]
    cu = s["cu_q"].long() if s["cu_q"] is not None else torch.arange(B + 1, device=dev)
    n = (cu[1:] - cu[:-1])[:, None]
    i = torch.arange(nq, device=dev)[None, :]
    row = torch.where(i < n, cu[:-1, None] + i, torch.full_like(i, rows))       # the row past the end: padding
    q = torch.cat((s["q"].float(), torch.zeros((1, hq * d), device=dev)))[row]  # [B, nq, hq * d]
    q = q.reshape(B, nq, hk, G, d).permute(0, 2, 3, 1, 4).reshape(B * hk, G * nq, d)
    K = cached("k")
    S = torch.matmul(q, K.transpose(1, 2).contiguous()) * (1.0 / math.sqrt(d))
    S = S.reshape(B, hk * G, nq, -1)
    del K
    pos = (lens - n + i)[:, :, None]                                            # [B, nq, 1]
    t = torch.arange(S.shape[-1], device=dev)[None, None, :]
    see = (t < lens[:, :, None]) & (pos >= 0)
    if c["causal"]:
        see = see & (t <= pos)
    if c["window"]:
        see = see & (t > pos - c["window"])
    see = see[:, None]
    S = S.masked_fill(~see, -math.inf)
    m = S.amax(-1, keepdim=True)
    P = torch.exp(S - torch.where(m == -math.inf, torch.zeros_like(m), m))
    del S
    l = P.sum(-1, keepdim=True)
    O = torch.matmul(P.reshape(B * hk, G * nq, -1), cached("v")).reshape(B, hk * G, nq, d)
    O = torch.where(l > 0, O / l, torch.zeros_like(O))             # a row that sees nothing is zero
    O = O.permute(0, 2, 1, 3).reshape(B * nq, hq * d).to(s["out"].dtype)
    out = torch.empty((rows + 1, hq * d), dtype=O.dtype, device=dev)
    out[row.reshape(-1)] = O
    s["out"].copy_(out[:rows])
    return {"out": s["out"]}


def _plain(s):
    op = s["case"]["op"]
    if op == "axes":
        for n in ("q", "k"):
            y = _norm_rope(s, s[n], s["gamma_" + n], torch.float32)
            s["out_" + n].copy_(_round(y.reshape(s[n].shape), s[n].dtype))
        return {"q": s["out_q"], "k": s["out_k"]}
    if op == "grad":
        for n in ("q", "k"):
            dx, dgamma = _plain_grad(s, s[n], s["dy_" + n], s["gamma_" + n])
            s["dx_" + n].copy_(dx)
            s["dgamma_" + n].copy_(dgamma)
        return {n: s[n] for n in ("dx_q", "dx_k", "dgamma_q", "dgamma_k")}
    return {"append": _plain_append, "gather": _plain_gather, "attend": _plain_attend}[op](s)


# ------------------------------------------------------------------ the framework's calls
def _calls(s):
    import layerwise_qk_norm_qknorm_amd as qk

    c = s["case"]
    op, d = c["op"], c["head_dim"]
    if op == "axes":
        q, k = qk.qknorm_headwise_rope_axes(s["q"], s["k"], s["gamma_q"], s["gamma_k"], EPS, d, s["cos_sin"],
                                            s["positions"], s["axes"], interleaved=c["interleaved"],
                                            gamma_head_stride=s["gamma_head_stride"], out_q=s["out_q"],
                                            out_k=s["out_k"])
        return {"q": q, "k": k}
    if op == "grad":
        got = qk.qknorm_headwise_rope_axes_backward(
            s["dy_q"], s["dy_k"], s["q"], s["k"], s["gamma_q"], s["gamma_k"], EPS, d, s["cos_sin"], s["positions"],
            s["axes"], interleaved=c["interleaved"], gamma_head_stride=s["gamma_head_stride"], dx_q=s["dx_q"],
            dx_k=s["dx_k"], dgamma_q=s["dgamma_q"], dgamma_k=s["dgamma_k"])
        return dict(zip(("dx_q", "dx_k", "dgamma_q", "dgamma_k"), got))
    if op == "append":
        rest = (s["k_cache"], s["v_cache"], s["slots"])
        kw = dict(k_scales=s["k_scales"], v_scales=s["v_scales"], interleaved=c["interleaved"], out_q=s["out_q"],
                  out_k=s["out_k"], out_v=s["out_v"])
        first = (s["q"], s["k"], s["v"], s["gamma_q"], s["gamma_k"], EPS, d, s["cos_sin"], s["positions"])
        if c["n_axes"]:
            q = qk.qknorm_paged_append_axes(*first, s["axes"], *rest, **kw)
        else:
            q = qk.qknorm_paged_append(*first, *rest, **kw)
        if c["cache"] == "rows":
            return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        return {"q": q, "k_values": s["out_k"], "v_values": s["out_v"]}
    if op == "gather":
        k, v = qk.qknorm_paged_gather(s["k_cache"], s["v_cache"], s["slots"], d, k_scales=s["k_scales"],
                                      v_scales=s["v_scales"], out_k=s["out_k"], out_v=s["out_v"])
        return {"k": k, "v": v}
    out = qk.qknorm_paged_attend_wide(s["q"], s["k_cache"], s["v_cache"], s["block_table"], s["seq_lens"], d,
                                      k_scales=s["k_scales"], v_scales=s["v_scales"], cu_q=s["cu_q"],
                                      causal=c["causal"], window=c["window"], max_q=s["max_q"],
                                      max_len=s["max_len"], out=s["out"])
    return {"out": out}


def run(state):
    return _calls(state) if own else _plain(state)


# ------------------------------------------------------------------ in 64 bits, from the definitions
def _rotated(x, s):
    """x [T, heads, d] float64 -> each pair (a, b) turned as the complex number a + ib, axis by axis."""
    c = s["case"]
    half = c["rot"] // 2
    turn = torch.zeros((x.shape[0], half), dtype=torch.complex128, device=x.device)
    pos = s["positions"].reshape(max(1, c["n_axes"]), -1)
    owner = torch.tensor(list(s["axes"]) if c["n_axes"] else [0] * half, device=x.device)
    for a in range(pos.shape[0]):
        row = s["cos_sin"].double()[pos[a]]
        turn = torch.where(owner == a, torch.complex(row[:, :half], row[:, half:]), turn)
    y = x.clone()
    i = torch.arange(half, device=x.device)
    first, second = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + half)
    z = torch.complex(x[..., first], x[..., second]) * turn[:, None, :]
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _defined(x, gamma, s):
    """Eq. 1 for every head, then the rotation; x and gamma float64."""
    d = s["case"]["head_dim"]
    x = x.reshape(x.shape[0], -1, d)
    if gamma is not None:
        eps = float(torch.tensor(EPS, dtype=torch.float32))
        rms = torch.sqrt(torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / d + eps)
        x = x / rms * gamma.reshape(-1, d)
    return _rotated(x, s)


def _magnitudes(cache, dev):
    """Every magnitude a code can have, by code."""
    if cache == "mxfp4":
        return torch.tensor(E2M1, dtype=torch.float64, device=dev)
    code = range(127)                                # 127 is NaN
    return torch.tensor([(n % 8) * 2.0 ** -9 if n < 8 else (8 + n % 8) * 2.0 ** (n // 8 - 10) for n in code],
                        dtype=torch.float64, device=dev)


def _nearest(x, cache):
    """x [..., d] float64 -> the values of the nearest codes, on a tie that of the even one."""
    _, top, lead = MX[cache]
    b = x.reshape(*x.shape[:-1], -1, 32)
    most = b.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(most))
    e = torch.where(torch.exp2(e) > most, e - 1, torch.where(torch.exp2(e + 1) <= most, e + 1, e)) - lead
    e = torch.where(most > 0, e, torch.full_like(e, LOWEST_EXPONENT)).clamp(LOWEST_EXPONENT, top)
    a = b.abs() * torch.exp2(-e)
    grid = _magnitudes(cache, x.device)
    hi = torch.searchsorted(grid, a.contiguous()).clamp(max=grid.numel() - 1)   # the first one not below
    lo = (hi - 1).clamp(min=0)
    up, down = (grid[hi] - a).abs(), (a - grid[lo]).abs()
    best = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), grid[hi], grid[lo])
    return (torch.sign(b) * best * torch.exp2(e)).reshape(x.shape)


def _stored(cache, codes, scales):
    """float64 values of a cache's entries, element by element from their codes."""
    if cache == "rows":
        return codes.double()
    grid = _magnitudes(cache, codes.device)
    if cache == "mxfp4":
        u = codes.int()
        n = torch.empty((*codes.shape[:-1], 2 * codes.shape[-1]), dtype=torch.int64, device=codes.device)
        n[..., 0::2], n[..., 1::2] = u % 16, u // 16
        x = grid[n % 8] * (1 - 2 * (n // 8))
    else:
        n = codes.long()
        x = grid[n % 128] * (1 - 2 * (n // 128))
    blocks = x.reshape(*x.shape[:-1], -1, 32) * torch.exp2(scales.double() - 127)[..., None]
    return blocks.reshape(x.shape)


def exact(c, seed):
    s = prepare(c, seed)
    op, d = c["op"], c["head_dim"]
    if op == "axes":
        top = 448.0 if c["dtype"] == "fp8" else math.inf
        return {n: _defined(s[n].double(), s["gamma_" + n].double(), s).reshape(s[n].shape).clamp(-top, top)
                for n in ("q", "k")}
    if op == "grad":
        out = {}
        for n in ("q", "k"):
            x = s[n].double().clone().requires_grad_()
            g = s["gamma_" + n].double().clone().requires_grad_()
            y = _defined(x, g, s).reshape(x.shape)
            out["dx_" + n], out["dgamma_" + n] = torch.autograd.grad(y, (x, g), s["dy_" + n].double())
        return out
    if op in ("append", "gather"):
        T, ps = c["T"], c["page"]
        kept = torch.nonzero(s["slots"] >= 0).reshape(-1)
        slot = s["slots"][kept]
    if op == "gather":
        got = {}
        for n in ("k", "v"):
            rows = s["out_" + n].double()
            at = (slot // ps, slice(None), slot % ps)
            scales = s[n + "_scales"]
            rows[kept] = _stored(c["cache"], s[n + "_cache"][at], None if scales is None else scales[at]).reshape(
                kept.numel(), -1)
            got[n] = rows
        return got
    if op == "append":
        g = [None if s["gamma_" + n] is None else s["gamma_" + n].double() for n in ("q", "k")]
        q = s["out_q"].double()
        q[kept] = _defined(s["q"].double(), g[0], s).reshape(T, -1)[kept]
        got = {"q": q}
        for n, x in (("k", _defined(s["k"].double(), g[1], s)), ("v", s["v"].double().reshape(T, -1, d))):
            if c["cache"] == "rows":
                flat = s[n + "_cache"].double().transpose(1, 2).contiguous()    # [pages, ps, heads, d]
                flat.reshape(-1, *flat.shape[2:])[slot] = x[kept]
                got[n + "_cache"] = flat.transpose(1, 2).contiguous()
            else:
                rows = s["out_" + n].double()
                rows[kept] = _nearest(x, c["cache"]).reshape(T, -1)[kept]
                got[n + "_values"] = rows
        return got
    if _visible(c)[1] * c["heads_q"] * d > 4e12:
        return None
    lens, nqs = _lengths(c)
    hq, hk, ps = c["heads_q"], c["heads_k"], c["page"]
    out = torch.zeros((sum(nqs), hq * d), dtype=torch.float64, device=s["q"].device)
    at = 0
    for b, (n, nq) in enumerate(zip(lens, nqs)):
        rows = slice(at, at + nq)
        at += nq
        if not n:
            continue
        pages = s["block_table"][b, :-(-n // ps)].long()
        i = torch.arange(n - nq, n, device=out.device)[:, None]
        t = torch.arange(n, device=out.device)[None, :]
        hidden = i < 0
        if c["causal"]:
            hidden = hidden | (t > i)
        if c["window"]:
            hidden = hidden | (i - t >= c["window"])
        for h in range(hk):
            kv = []
            for name in ("k", "v"):
                scales = s[name + "_scales"]
                x = _stored(c["cache"], s[name + "_cache"][pages, h], None if scales is None else scales[pages, h])
                kv.append(x.reshape(-1, d)[:n])
            for j in range(h * (hq // hk), (h + 1) * (hq // hk)):
                score = s["q"][rows, j * d:(j + 1) * d].double() @ kv[0].t() / math.sqrt(d)
                score = score.masked_fill(hidden, -math.inf)
                p = torch.nan_to_num(torch.softmax(score, -1))      # a row that sees nothing
                out[rows, j * d:(j + 1) * d] = p @ kv[1]
    return {"out": out}

"""The operators with several axes and wide caches as they are used together: prompts of images and
text appended and attended to, chunk by chunk, then decode steps and a prefix read back; graphs,
streams, prepared calls; a training step's graph."""

import numpy as np
import pytest
import torch

import layerwise_qk_norm_qknorm_amd as qk
import operator_cases as C
from oracle import operators as O

pytestmark = pytest.mark.gpu
EPS = 1e-6
D, HQ, HK, PS = 128, 10, 2, 16
AXES = bytes([0] * 16 + [1] * 24 + [2] * 24)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qk.load_library()
    yield
    torch.cuda.synchronize()


class Server:
    """A cache, its block table and the weights of one attention layer's norms."""

    def __init__(self, fmt, B, pages=64):
        r = C.rng(7)
        self.fmt = fmt
        if fmt == "rows":
            self.cache = [torch.randint(-30000, 30000, (pages, HK, PS, D), device="cuda").short().view(torch.bfloat16)
                          for _ in range(2)]
            self.scales = {}
        else:
            self.cache = [torch.randint(0, 256, (pages, HK, PS, D), device="cuda").byte() for _ in range(2)]
            s = [torch.randint(0, 256, (pages, HK, PS, D // 32), device="cuda").byte() for _ in range(2)]
            self.scales = dict(k_scales=s[0], v_scales=s[1])
        self.table = torch.from_numpy(r.permutation(pages).reshape(B, -1).astype(np.int32)).cuda()
        self.gq = C.dev(C.to_type(r.normal(1, 0.1, D), "bf16"))
        self.gk = C.dev(C.to_type(r.normal(1, 0.1, D), "bf16"))
        self.cos_sin = qk.rope_table(1024, D)
        self.lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.rows = [[[] for _ in range(B)] for _ in range(2)]

    def slots(self, b, pos):
        return self.table[b.long(), (pos // PS)].long() * PS + pos % PS

    def step(self, qkv, n_new):
        """qkv rows of n_new tokens per sequence -> attention output; checked against the oracle
        on what the gather reads back."""
        B = len(n_new)
        b = torch.cat([torch.full((n,), i, device="cuda") for i, n in enumerate(n_new)])
        place = torch.cat([torch.arange(n, device="cuda") + int(self.lens[i]) for i, n in enumerate(n_new)])
        pos = torch.stack((place // 20, place % 20 // 5, place % 5))         # frames of four rows of five
        q, k, v = qkv[:, :HQ * D], qkv[:, HQ * D:(HQ + HK) * D], qkv[:, (HQ + HK) * D:]
        ok, ov = torch.empty_like(k), torch.empty_like(v)
        slots = self.slots(b, place)
        qn = qk.qknorm_paged_append_axes(q, k, v, self.gq, self.gk, EPS, D, self.cos_sin, pos, AXES, *self.cache, slots,
                                         out_q=torch.empty_like(q), out_k=ok, out_v=ov, **self.scales)
        self.lens += torch.tensor(n_new, dtype=torch.int32, device="cuda")
        cu = np.concatenate(([0], np.cumsum(n_new))).astype(np.int32)
        out = qk.qknorm_paged_attend_wide(qn, *self.cache, self.table, self.lens, D,
                                          cu_q=None if max(n_new) == 1 and min(n_new) == 1 else C.dev(cu),
                                          max_q=max(n_new), **self.scales)
        back = qk.qknorm_paged_gather(*self.cache, slots, D, **self.scales)
        torch.cuda.synchronize()
        assert C.same_bits(back[0], ok) and C.same_bits(back[1], ov)
        got = C.host_values(out).reshape(-1, HQ, D)
        for i in range(B):
            rows = slice(cu[i], cu[i + 1])
            KV = []
            for held, t in zip(self.rows, back):
                held[i].append(C.host_values(t[rows]))
                KV.append(np.concatenate(held[i]).reshape(-1, HK, D))
            want, mag, _ = O.attend(C.host_values(qn[rows]).reshape(-1, HQ, D), *KV, n_new[i], D ** -0.5, True, 0)
            C.close(got[rows], want, 2.0 ** -8 * np.abs(want) + 2.0 ** -7 * mag, f"sequence {i}")


@pytest.mark.parametrize("fmt", ["rows", "mxfp8"])
def test_prompts_in_chunks_then_decode_steps(fmt):
    s = Server(fmt, 4)
    g = torch.Generator(device="cuda").manual_seed(3)

    def rows(n):
        return torch.randn((n, (HQ + 2 * HK) * D), generator=g, device="cuda").bfloat16()

    for n in ([37, 5, 100, 1], [60, 1, 1, 50]):            # prompts, then a mixed step: chunks and decodes
        s.step(rows(sum(n)), n)
    for _ in range(3):
        s.step(rows(4), [1, 1, 1, 1])


def _everything(w):
    """One of each call on preallocated memory."""
    q, k, v = w["q"], w["k"], w["v"]
    a = (EPS, D, w["table"], w["pos"], AXES)
    qk.qknorm_headwise_rope_axes(q, k, w["gq"], w["gk"], *a, out_q=w["yq"], out_k=w["yk"])
    qk.qknorm_headwise_rope_axes_backward(w["yq"], w["yk"], q, k, w["gq"], w["gk"], *a, dx_q=w["dq"], dx_k=w["dk"],
                                          dgamma_q=w["dgq"], dgamma_k=w["dgk"])
    qk.qknorm_paged_append_axes(q, k, v, w["gq"], w["gk"], *a, w["kc"], w["vc"], w["slots"], w["ks"], w["vs"],
                                out_q=w["aq"])
    qk.qknorm_paged_gather(w["kc"], w["vc"], w["slots"], D, w["ks"], w["vs"], out_k=w["kr"], out_v=w["vr"])
    w["kb"][:, :, :].copy_(w["kr"].view(-1, PS, HK, D).transpose(1, 2))
    w["vb"][:, :, :].copy_(w["vr"].view(-1, PS, HK, D).transpose(1, 2))
    qk.qknorm_paged_attend_wide(w["aq"], w["kc"], w["vc"], w["bt"], w["lens"], D, w["ks"], w["vs"], cu_q=w["cu"],
                                max_q=w["T"], out=w["o"])
    qk.qknorm_paged_attend_wide(w["aq"][-1:], w["kb"], w["vb"], w["bt"], w["lens"], D, out=w["o1"])     # split, joined


def _world(T=640, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((T, (HQ + 2 * HK) * D), generator=g, device="cuda").bfloat16()
    w = {"T": T, "x": x, "q": x[:, :HQ * D], "k": x[:, HQ * D:(HQ + HK) * D], "v": x[:, (HQ + HK) * D:]}
    w["table"] = qk.rope_table(T, D)
    i = torch.arange(T, device="cuda")
    w["pos"] = torch.stack((i // 64, i % 64 // 8, i % 8))
    w["gq"], w["gk"] = (torch.rand(D, generator=g, device="cuda").bfloat16() + 0.5 for _ in range(2))
    for n, like in (("yq", "q"), ("yk", "k"), ("dq", "q"), ("dk", "k"), ("aq", "q"), ("o", "q"), ("kr", "k"), ("vr", "k")):
        w[n] = torch.zeros((T, w[like].shape[1]), dtype=torch.bfloat16, device="cuda")
    w["o1"] = torch.zeros((1, HQ * D), dtype=torch.bfloat16, device="cuda")
    w["dgq"], w["dgk"] = (torch.zeros(D, device="cuda") for _ in range(2))
    pages = T // PS
    for n, last in (("kc", D), ("vc", D), ("ks", D // 32), ("vs", D // 32)):
        w[n] = torch.zeros((pages, HK, PS, last), dtype=torch.uint8, device="cuda")
    for n in ("kb", "vb"):
        w[n] = torch.zeros((pages, HK, PS, D), dtype=torch.bfloat16, device="cuda")
    w["bt"] = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    w["slots"] = i.clone()
    w["lens"] = torch.tensor([T], dtype=torch.int32, device="cuda")
    w["cu"] = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    return w


OUTS = ("yq", "yk", "dq", "dk", "dgq", "dgk", "kc", "vc", "ks", "vs", "aq", "kr", "vr", "o", "o1")


def test_graph_replays_equal_eager_calls():
    w, ref = _world(seed=1), _world(seed=1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _everything(w)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        _everything(w)
    for rep in range(4):
        new = torch.randn(w["x"].shape, generator=torch.Generator(device="cuda").manual_seed(50 + rep),
                          device="cuda").bfloat16()
        for z in (w, ref):
            z["x"].copy_(new)
            for n in OUTS:
                z[n].zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        _everything(ref)
        torch.cuda.synchronize()
        for n in OUTS:
            assert C.same_bits(w[n], ref[n]), (rep, n)
        assert w["o"].float().abs().max() > 0 and w["o1"].float().abs().max() > 0


def test_two_streams_at_once_and_a_stream_that_is_not_current():
    a, b, ref = _world(seed=2), _world(seed=3), [_world(seed=2), _world(seed=3)]
    for r in ref:
        _everything(r)
    torch.cuda.synchronize()
    s = [torch.cuda.Stream() for _ in range(2)]
    for st in s:
        st.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for st, w in zip(s, (a, b)):
            with torch.cuda.stream(st):
                _everything(w)
    torch.cuda.synchronize()
    for w, r in zip((a, b), ref):
        for n in OUTS:
            assert C.same_bits(w[n], r[n]), n
    # outputs and workspaces that the call allocates belong to the stream it is given
    for stream in (s[0], s[0].cuda_stream, 0):
        o = [qk.qknorm_paged_attend_wide(a["aq"][-1:], a["kb"], a["vb"], a["bt"], a["lens"], D, stream=stream)
             for _ in range(3)]
        k = [qk.qknorm_paged_gather(a["kc"], a["vc"], a["slots"], D, a["ks"], a["vs"], stream=stream) for _ in range(3)]
        g = [qk.qknorm_headwise_rope_axes_backward(a["yq"], a["yk"], a["q"], a["k"], a["gq"], a["gk"], EPS, D,
                                                   a["table"], a["pos"], AXES, stream=stream) for _ in range(3)]
        torch.cuda.synchronize()
        for x in o:
            assert C.same_bits(x, a["o1"])
        for x in k:
            assert C.same_bits(x[0], a["kr"]) and C.same_bits(x[1], a["vr"])
        for x in g:
            assert C.same_bits(x[0], a["dq"]) and C.same_bits(x[2], a["dgq"])


def test_prepared_calls_equal_the_plain_ones():
    w, p = _world(seed=4), _world(seed=4)
    a = (EPS, D, p["table"], p["pos"], AXES)
    calls = [
        qk.prepare_headwise_rope_axes(p["q"], p["k"], p["gq"], p["gk"], *a, out_q=p["yq"], out_k=p["yk"]),
        qk.prepare_headwise_rope_axes_backward(p["yq"], p["yk"], p["q"], p["k"], p["gq"], p["gk"], *a, dx_q=p["dq"],
                                               dx_k=p["dk"], dgamma_q=p["dgq"], dgamma_k=p["dgk"]),
        qk.prepare_paged_append_axes(p["q"], p["k"], p["v"], p["gq"], p["gk"], *a, p["kc"], p["vc"], p["slots"], p["ks"],
                                     p["vs"], out_q=p["aq"]),
        qk.prepare_paged_gather(p["kc"], p["vc"], p["slots"], D, p["ks"], p["vs"], out_k=p["kr"], out_v=p["vr"]),
        lambda: (p["kb"].copy_(p["kr"].view(-1, PS, HK, D).transpose(1, 2)),
                 p["vb"].copy_(p["vr"].view(-1, PS, HK, D).transpose(1, 2))),
        qk.prepare_paged_attend_wide(p["aq"], p["kc"], p["vc"], p["bt"], p["lens"], D, p["ks"], p["vs"], cu_q=p["cu"],
                                     max_q=p["T"], out=p["o"]),
        qk.prepare_paged_attend_wide(p["aq"][-1:], p["kb"], p["vb"], p["bt"], p["lens"], D, out=p["o1"]),
    ]
    side = torch.cuda.Stream()
    for rep in range(3):
        if rep:
            for z in (w, p):
                z["x"].mul_(-1.5)
        _everything(w)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side if rep == 2 else torch.cuda.current_stream()):
            for c in calls:
                c()
        torch.cuda.synchronize()
        for n in OUTS:
            assert C.same_bits(w[n], p[n]), (rep, n)
    made = qk.prepare_paged_gather(w["kc"], w["vc"], w["slots"], D, w["ks"], w["vs"])      # its own rows
    k, v = made()
    torch.cuda.synchronize()
    assert C.same_bits(k, w["kr"]) and C.same_bits(v, w["vr"])


def test_a_training_step_as_an_autograd_function():
    """Forward and backward as a module uses them, and the two calls captured into a graph."""
    T = 200

    class Turn(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k, gq, gk, table, pos):
            ctx.save_for_backward(q, k, gq, gk, table, pos)
            oq, ok = torch.empty_like(q), torch.empty_like(k)
            return qk.qknorm_headwise_rope_axes(q, k, gq, gk, EPS, D, table, pos, AXES, out_q=oq, out_k=ok)

        @staticmethod
        def backward(ctx, dq, dk):
            q, k, gq, gk, table, pos = ctx.saved_tensors
            dx = qk.qknorm_headwise_rope_axes_backward(dq.contiguous(), dk.contiguous(), q, k, gq, gk, EPS, D, table, pos,
                                                       AXES)
            return (*dx, None, None)

    g = torch.Generator(device="cuda").manual_seed(9)
    q, k = (torch.randn((T, h * D), generator=g, device="cuda", requires_grad=True) for h in (HQ, HK))
    gq, gk = (torch.rand(D, generator=g, device="cuda", requires_grad=True) for _ in range(2))
    table = qk.rope_table(64, D)
    pos = torch.randint(0, 64, (3, T), generator=g, device="cuda")
    u = [torch.randn((T, h * D), generator=g, device="cuda") for h in (HQ, HK)]
    leaves = (q, k, gq, gk)

    def loss():
        y = Turn.apply(q, k, gq, gk, table, pos)
        return (y[0] * u[0]).sum() + (y[1] * u[1]).sum()

    eager = torch.autograd.grad(loss(), leaves)
    wg = O.norm_rope_backward(q.detach().cpu().numpy(), u[0].cpu().numpy(), gq.detach().cpu().numpy(), EPS, D, 0,
                              *O.axis_angles(table.cpu().numpy(), pos.cpu().numpy(), AXES, D), False)
    C.close(eager[0].cpu().numpy().astype(np.float64).reshape(wg[0].shape), wg[0], wg[2] * 120 * C.U, "dx")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(loss(), leaves)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = Turn.apply(q.detach(), k.detach(), gq.detach(), gk.detach(), table, pos)
        captured = qk.qknorm_headwise_rope_axes_backward(u[0], u[1], q.detach(), k.detach(), gq.detach(), gk.detach(),
                                                         EPS, D, table, pos, AXES)
    for _ in range(3):
        for t in captured + tuple(y):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(captured, eager):
            assert C.same_bits(a, b)

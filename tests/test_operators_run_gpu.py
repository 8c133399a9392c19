"""The operators as they are used together: prompts appended and read back by
attention, then decode steps; a training step's forward and backward; graphs,
streams and prepared calls."""

import numpy as np
import pytest
import torch

import layerwise_qk_norm_qknorm_amd as qk
import operator_cases as C
from oracle import operators as O

pytestmark = pytest.mark.gpu
EPS = 1e-6
D, HQ, HK, PS = 128, 10, 2, 16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qk.load_library()
    yield
    torch.cuda.synchronize()


class Server:
    """A cache, its block table and the weights of one attention layer's norms."""

    def __init__(self, B, pages=64):
        r = C.rng(7)
        self.kc, self.vc = (torch.randint(0, 256, (pages, HK, PS, D // 2), device="cuda").byte() for _ in range(2))
        self.ks, self.vs = (torch.randint(0, 256, (pages, HK, PS, D // 32), device="cuda").byte() for _ in range(2))
        self.table = torch.from_numpy(r.permutation(pages).reshape(B, -1).astype(np.int32)).cuda()
        self.gq = C.dev(C.to_type(r.normal(1, 0.1, D), "bf16"))
        self.gk = C.dev(C.to_type(r.normal(1, 0.1, D), "bf16"))
        self.cos_sin = qk.rope_table(1024, D)
        self.lens = torch.zeros(B, dtype=torch.int32, device="cuda")
        self.k_rows = [[] for _ in range(B)]
        self.v_rows = [[] for _ in range(B)]

    def slots(self, b, pos):
        return self.table[b.long(), (pos // PS)].long() * PS + pos % PS

    def step(self, qkv, n_new):
        """qkv rows of n_new tokens per sequence -> attention output; checked against the oracle
        on the values the cache says it holds."""
        B = len(n_new)
        b = torch.cat([torch.full((n,), i, device="cuda") for i, n in enumerate(n_new)])
        pos = torch.cat([torch.arange(n, device="cuda") + int(self.lens[i]) for i, n in enumerate(n_new)])
        q, k, v = qkv[:, :HQ * D], qkv[:, HQ * D:(HQ + HK) * D], qkv[:, (HQ + HK) * D:]
        ok, ov = torch.empty_like(k), torch.empty_like(v)
        qn = qk.qknorm_paged_append(q, k, v, self.gq, self.gk, EPS, D, self.cos_sin, pos, self.kc, self.vc,
                                    self.slots(b, pos), self.ks, self.vs, out_q=torch.empty_like(q), out_k=ok,
                                    out_v=ov)
        self.lens += torch.tensor(n_new, dtype=torch.int32, device="cuda")
        cu = np.concatenate(([0], np.cumsum(n_new))).astype(np.int32)
        out = qk.qknorm_paged_attend(qn, self.kc, self.vc, self.ks, self.vs, self.table, self.lens, D,
                                     cu_q=None if max(n_new) == 1 and min(n_new) == 1 else C.dev(cu),
                                     max_q=max(n_new))
        torch.cuda.synchronize()
        got = C.host_values(out).reshape(-1, HQ, D)
        for i in range(B):
            rows = slice(cu[i], cu[i + 1])
            self.k_rows[i].append(C.host_values(ok[rows]))
            self.v_rows[i].append(C.host_values(ov[rows]))
            K = np.concatenate(self.k_rows[i]).reshape(-1, HK, D)
            V = np.concatenate(self.v_rows[i]).reshape(-1, HK, D)
            want, mag, _ = O.attend(C.host_values(qn[rows]).reshape(-1, HQ, D), K, V, n_new[i], D ** -0.5, True, 0)
            C.close(got[rows], want, 2.0 ** -8 * np.abs(want) + 2.0 ** -7 * mag, f"sequence {i}")
        return out


def test_prompts_then_decode_steps():
    s = Server(4)
    g = torch.Generator(device="cuda").manual_seed(3)

    def rows(n):
        return torch.randn((n, (HQ + 2 * HK) * D), generator=g, device="cuda").bfloat16()

    n = [37, 5, 100, 1]
    s.step(rows(sum(n)), n)            # prompts
    n = [20, 1, 1, 50]
    s.step(rows(sum(n)), n)            # a mixed step: chunks and decodes
    for _ in range(3):
        s.step(rows(4), [1, 1, 1, 1])  # decode


def test_a_layerwise_norm_goes_before_the_append():
    """qknorm_fused over the whole vectors, then the append without gamma: K rotated only."""
    T = 33
    x = C.dev(C.to_type(C.rng(1).normal(size=(T, (HQ + 2 * HK) * D)), "bf16"))
    q, k, v = x[:, :HQ * D], x[:, HQ * D:(HQ + HK) * D], x[:, (HQ + HK) * D:]
    gq, gk = torch.ones(HQ * D, device="cuda").bfloat16(), torch.ones(HK * D, device="cuda").bfloat16()
    qk.qknorm_fused(q, k, gq, gk, EPS)
    kc, vc = (torch.zeros((4, HK, PS, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pos = torch.arange(T, device="cuda")
    table = qk.rope_table(64, D)
    want_k = torch.empty_like(k)
    norm = C.values(C.torch_to_np(k))
    qk.qknorm_paged_append(q, k, v, None, None, EPS, D, table, pos, kc, vc, pos + 16, out_k=want_k)
    torch.cuda.synchronize()
    cos, sin = O.angles(table.cpu().numpy(), np.arange(T), D)
    z = norm.reshape(T, HK, D)
    C.close(C.host_values(want_k).reshape(z.shape), O.rotate(z, cos, sin, False), C.rope_bound(z, cos, sin, False, "bf16"),
            "k")
    assert torch.equal(kc[1:3].transpose(1, 2).reshape(32, -1), want_k[:32])
    assert torch.equal(vc[1:3].transpose(1, 2).reshape(32, -1), v[:32])


def _everything(w):
    """One of each call on preallocated memory."""
    q, k, v = w["q"], w["k"], w["v"]
    a = (EPS, D, w["table"], w["pos"])
    qk.qknorm_headwise_rope(q, k, w["gq"], w["gk"], *a, out_q=w["yq"], out_k=w["yk"])
    qk.qknorm_headwise_rope_backward(w["yq"], w["yk"], q, k, w["gq"], w["gk"], *a, dx_q=w["dq"], dx_k=w["dk"],
                                     dgamma_q=w["dgq"], dgamma_k=w["dgk"])
    qk.qknorm_paged_append(q, k, v, w["gq"], w["gk"], *a, w["kc"], w["vc"], w["slots"], w["ks"], w["vs"],
                           out_q=w["aq"])
    qk.qknorm_paged_attend(w["aq"], w["kc"], w["vc"], w["ks"], w["vs"], w["bt"], w["lens"], D, cu_q=w["cu"],
                           max_q=w["T"], out=w["o"])


def _world(T=600, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((T, (HQ + 2 * HK) * D), generator=g, device="cuda").bfloat16()
    w = {"T": T, "x": x, "q": x[:, :HQ * D], "k": x[:, HQ * D:(HQ + HK) * D], "v": x[:, (HQ + HK) * D:]}
    w["table"], w["pos"] = qk.rope_table(T, D), torch.arange(T, device="cuda")
    w["gq"], w["gk"] = (torch.rand(D, generator=g, device="cuda").bfloat16() + 0.5 for _ in range(2))
    for n, like in (("yq", "q"), ("yk", "k"), ("dq", "q"), ("dk", "k"), ("aq", "q"), ("o", "q")):
        w[n] = torch.zeros((T, w[like].shape[1]), dtype=torch.bfloat16, device="cuda")
    w["dgq"], w["dgk"] = (torch.zeros(D, device="cuda") for _ in range(2))
    pages = T // PS + 1
    for n, last in (("kc", D // 2), ("vc", D // 2), ("ks", D // 32), ("vs", D // 32)):
        w[n] = torch.zeros((pages, HK, PS, last), dtype=torch.uint8, device="cuda")
    w["bt"] = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    w["slots"] = w["pos"].clone()
    w["lens"] = torch.tensor([T], dtype=torch.int32, device="cuda")
    w["cu"] = torch.tensor([0, T], dtype=torch.int32, device="cuda")
    return w


OUTS = ("yq", "yk", "dq", "dk", "dgq", "dgk", "kc", "vc", "ks", "vs", "aq", "o")


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
        assert w["o"].float().abs().max() > 0


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
    for stream in (s[0], s[0].cuda_stream):
        o = [qk.qknorm_paged_attend(a["aq"], a["kc"], a["vc"], a["ks"], a["vs"], a["bt"], a["lens"], D, cu_q=a["cu"],
                                    max_q=1, stream=stream) for _ in range(3)]
        g = [qk.qknorm_headwise_rope_backward(a["yq"], a["yk"], a["q"], a["k"], a["gq"], a["gk"], EPS, D, a["table"],
                                              a["pos"], stream=stream) for _ in range(3)]
        torch.cuda.synchronize()
        for x in o:
            assert C.same_bits(x, o[0])
        for x in g:
            assert C.same_bits(x[0], a["dq"]) and C.same_bits(x[2], a["dgq"])


def test_prepared_calls_equal_the_plain_ones():
    w, p = _world(seed=4), _world(seed=4)
    a = (EPS, D, p["table"], p["pos"])
    calls = [
        qk.prepare_headwise_rope(p["q"], p["k"], p["gq"], p["gk"], *a, out_q=p["yq"], out_k=p["yk"]),
        qk.prepare_headwise_rope_backward(p["yq"], p["yk"], p["q"], p["k"], p["gq"], p["gk"], *a, dx_q=p["dq"],
                                          dx_k=p["dk"], dgamma_q=p["dgq"], dgamma_k=p["dgk"]),
        qk.prepare_paged_append(p["q"], p["k"], p["v"], p["gq"], p["gk"], *a, p["kc"], p["vc"], p["slots"], p["ks"],
                                p["vs"], out_q=p["aq"]),
        qk.prepare_paged_attend(p["aq"], p["kc"], p["vc"], p["ks"], p["vs"], p["bt"], p["lens"], D, cu_q=p["cu"],
                                max_q=p["T"], out=p["o"]),
    ]
    for rep in range(2):
        if rep:
            for z in (w, p):
                z["x"].mul_(-1.5)
        _everything(w)
        for c in calls:
            c()
        torch.cuda.synchronize()
        for n in OUTS:
            assert C.same_bits(w[n], p[n]), n


def test_gradients_against_differences_of_the_forward_call():
    """A directional difference of the float32 forward call: (f(x + h u) - f(x - h u)) / 2h
    against dx . u. With h = 2^-6 and unit-scale data the third-order term and float32 rounding of
    about 3e4 outputs stay below 1% of the terms' root sum of squares."""
    T = 12
    r = C.rng(5)
    x = r.normal(size=(T, (HQ + HK) * D))
    u, dy = r.normal(size=x.shape), r.normal(size=x.shape)
    gq, gk = (torch.rand(D, device="cuda") + 0.5 for _ in range(2))
    table, pos = qk.rope_table(100, D), torch.arange(T, device="cuda") * 3

    def split(a):
        t = torch.from_numpy(a.astype(np.float32)).cuda()
        return t[:, :HQ * D], t[:, HQ * D:]

    def f(a):
        q, k = split(a)
        oq, ok = qk.qknorm_headwise_rope(q, k, gq, gk, EPS, D, table, pos)
        return np.concatenate((oq.cpu().numpy(), ok.cpu().numpy()), 1).astype(np.float64)

    q, k = split(x)
    dq, dk = split(dy)
    got = qk.qknorm_headwise_rope_backward(dq, dk, q, k, gq, gk, EPS, D, table, pos)
    dx = np.concatenate((got[0].cpu().numpy(), got[1].cpu().numpy()), 1).astype(np.float64)
    h = 2.0 ** -6
    lhs = ((f(x + h * u) - f(x - h * u)) / (2 * h) * dy).sum()
    assert abs(lhs - (dx * u).sum()) < 0.01 * np.sqrt((dx * dx).sum())

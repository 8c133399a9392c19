"""qknorm_paged_attend on ragged batches whose longest sequence the caller does not name: the
call without max_q gives the bits of the call with it, and agrees with the float64 oracle."""

import numpy as np
import pytest
import torch

import layerwise_qk_norm_qknorm_amd as qk
import operator_cases as C
from oracle import operators as O

pytestmark = pytest.mark.gpu
D, HQ, HK, PS = 128, 40, 8, 16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qk.load_library()
    yield
    torch.cuda.synchronize()
    torch.cuda.empty_cache()


@pytest.mark.parametrize("kind,B,T", [("even", 256, 120000), ("even", 512, 60000), ("even", 4096, 8192),
                                      ("one long", 300, 3300)])
def test_without_a_bound_on_the_rows(kind, B, T):
    print(f"[case] ragged {kind} {B} {T}", flush=True)
    r = C.rng(B)
    if kind == "even":
        n_q = r.multinomial(T - B, np.full(B, 1 / B)) + 1
    else:
        n_q = np.ones(B, np.int64)
        n_q[B // 3] = T - B + 1
    lens = n_q + r.integers(0, 40, B)
    need = -(-lens // PS)
    pages = int(need.sum())
    first = np.concatenate(([0], np.cumsum(need)))
    order = r.permutation(pages).astype(np.int32)
    table = np.zeros((B, int(need.max())), np.int32)
    for b in range(B):
        table[b, :need[b]] = order[first[b]:first[b + 1]]
    g = torch.Generator(device="cuda").manual_seed(B)
    codes = [torch.randint(0, 256, (pages, HK, PS, D // 2), generator=g, device="cuda").byte() for _ in range(2)]
    scales = [torch.randint(124, 128, (pages, HK, PS, D // 32), generator=g, device="cuda").byte() for _ in range(2)]
    q = torch.randn((T, HQ * D), generator=g, device="cuda", dtype=torch.bfloat16)
    cu = np.concatenate(([0], np.cumsum(n_q))).astype(np.int32)
    args = (q, *codes, *scales, C.dev(table), C.dev(lens.astype(np.int32)), D)
    out = qk.qknorm_paged_attend(*args, cu_q=C.dev(cu))
    same = qk.qknorm_paged_attend(*args, cu_q=C.dev(cu), max_q=int(n_q.max()), max_len=int(lens.max()))
    torch.cuda.synchronize()
    if n_q.max() * HQ // HK > 32:       # both calls take four row tiles a block
        assert C.same_bits(out, same)
    for b in {0, 1, B // 3, B // 2, B - 1}:
        n, rows = int(lens[b]), slice(int(cu[b]), int(cu[b + 1]))
        at = torch.from_numpy(table[b, :need[b]]).cuda().long()
        k, v = (O.mxfp4_values(c[at].cpu().numpy(), s[at].cpu().numpy()).transpose(0, 2, 1, 3)
                .reshape(-1, HK, D)[:n] for c, s in zip(codes, scales))
        if n_q[b] > 40:     # the first and the last rows of a long sequence
            keep = np.r_[0:8, n_q[b] - 8:n_q[b]]
        else:
            keep = np.arange(n_q[b])
        qv = C.host_values(q[rows]).reshape(-1, HQ, D)
        for i in keep:
            end = n - int(n_q[b]) + int(i) + 1
            want, mag, _ = O.attend(qv[i:i + 1], k[:end], v[:end], 1, D ** -0.5, True, 0)
            for o in (out, same):
                got = C.host_values(o[rows][i:i + 1]).reshape(1, HQ, D)
                # the tolerance of test_paged_attend_gpu.py
                C.close(got, want, 2.0 ** -8 * np.abs(want) + 2.0 ** -7 * mag + 2.0 ** -134, f"{b} {i}")

"""Calls of the rotation and the append that a capped grid takes in many passes: run here and
in a child process under QKNORM_MAX_GRID, whose outputs are compared bit for bit.

    QKNORM_MAX_GRID=7 python tests/operator_cap_cases.py OUT.npz
"""

import os
import sys

if __name__ == "__main__":
    HERE = os.path.dirname(os.path.abspath(__file__))
    sys.path[:0] = [os.path.dirname(HERE), HERE]

import numpy as np
import torch

# call, row type, tokens, query and key heads, head width, interleaved
CASES = [
    ("rope", "bf16", 900, 10, 2, 128, False),
    ("rope", "f32", 333, 5, 1, 128, True),
    ("rope", "fp8", 700, 4, 4, 64, False),
    ("rope", "bf16", 500, 9, 3, 80, False),
    ("rope", "bf16", 200, 40, 8, 320, False),       # three blocks a token
    ("rope", "f32", 150, 3, 2, 33, False),
    ("mxfp4", "bf16", 900, 10, 2, 128, False),
    ("mxfp4", "bf16", 2500, 10, 2, 128, True),
    ("mxfp4", "bf16", 300, 6, 2, 96, False),
    ("rows", "bf16", 900, 10, 2, 128, False),
    ("rows", "bf16", 300, 6, 2, 80, False),
]


def run(case):
    """The call's outputs as arrays of bytes."""
    import layerwise_qk_norm_qknorm_amd as qk
    import operator_cases as C
    call, dtype, T, nq, nk, d, inter = case
    r = C.rng(T + d)
    rot = d - d % 2
    x = C.dev(C.to_type(r.normal(size=(T, (nq + 2 * nk) * d)), dtype))
    q, k, v = x[:, :nq * d], x[:, nq * d:(nq + nk) * d], x[:, (nq + nk) * d:]
    g = [C.dev(C.to_type(r.normal(1, 0.2, size=d), "bf16" if dtype == "fp8" else dtype)) for _ in range(2)]
    tab, pos = C.dev(C.table(600, rot)), C.dev(r.integers(0, 600, T))
    oq = torch.zeros((T, nq * d), dtype=x.dtype, device="cuda")
    if call == "rope":
        ok = torch.zeros((T, nk * d), dtype=x.dtype, device="cuda")
        qk.qknorm_headwise_rope(q, k, *g, 1e-6, d, tab, pos, inter, 0, oq, ok)
        out = (oq, ok)
    else:
        ps, pages = 16, T // 16 + 2
        four = call == "mxfp4"
        cache = [torch.zeros((pages, nk, ps, d // 2 if four else d), dtype=torch.uint8 if four else x.dtype,
                             device="cuda") for _ in range(2)]
        scales = [torch.zeros((pages, nk, ps, d // 32), dtype=torch.uint8, device="cuda") if four else None
                  for _ in range(2)]
        slots = r.permutation(pages * ps)[:T].astype(np.int64)
        slots[5] = -1
        qk.qknorm_paged_append(q, k, v, *g, 1e-6, d, tab, pos, *cache, C.dev(slots), *scales, inter, out_q=oq)
        out = (oq, *cache, *(s for s in scales if s is not None))
    torch.cuda.synchronize()
    return [t.contiguous().view(torch.uint8).cpu().numpy() for t in out]


def main(path):
    res = {}
    for i, case in enumerate(CASES):
        print(f"[child] cap {os.environ.get('QKNORM_MAX_GRID')} {case}", flush=True)
        for n, a in enumerate(run(case)):
            res[f"{i}_{n}"] = a
    np.savez(path, **res)
    print("[child] done", flush=True)


if __name__ == "__main__":
    main(sys.argv[1])

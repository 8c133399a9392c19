"""QKNORM_MAX_GRID and the operators around headwise QK-Norm: with seven blocks to a launch every
block takes many tokens, and results equal those of the uncapped calls bit for bit."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import layerwise_qk_norm_qknorm_amd as qk
from operator_cap_cases import CASES, run

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def capped(tmp_path_factory):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    assert "QKNORM_MAX_GRID" not in os.environ, "the uncapped calls need the variable unset"
    qk.load_library()
    out = str(tmp_path_factory.mktemp("cap") / "capped.npz")
    res = subprocess.run([sys.executable, "-u", os.path.join(HERE, "operator_cap_cases.py"), out],
                         env=dict(os.environ, QKNORM_MAX_GRID="7"), capture_output=True, text=True, timeout=200)
    print(res.stdout[-2000:], res.stderr[-2000:], flush=True)
    assert res.returncode == 0, f"child process failed ({res.returncode})"
    with np.load(out) as d:
        return {k: d[k] for k in d.files}


@pytest.mark.parametrize("i", range(len(CASES)), ids=lambda i: "-".join(str(x) for x in CASES[i]))
def test_capped_grids_give_the_same_bits(i, capped):
    print(f"[case] cap {CASES[i]}", flush=True)
    for n, a in enumerate(run(CASES[i])):
        assert np.array_equal(a, capped[f"{i}_{n}"]), n

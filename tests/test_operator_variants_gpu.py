"""The operators' less ordinary kernel variants (operator_variants.py), by the tests that the
ordinary ones go through."""

import pytest
import torch

import layerwise_qk_norm_qknorm_amd as qk
import test_paged_append_gpu as A
import test_rope_gpu as R
from operator_variants import APPEND, ROPE

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    qk.load_library()
    yield
    torch.cuda.synchronize()


def _name(c):
    return "-".join(str(x) for x in (c.values() if isinstance(c, dict) else c))


@pytest.mark.parametrize("case", [c for c, _ in ROPE], ids=_name)
def test_forward(case):
    R.test_forward_against_the_oracle(case)


@pytest.mark.parametrize("case", [c for c, _ in ROPE if c[0] != "fp8"], ids=_name)
def test_backward(case):
    R.test_backward_against_the_oracle(case)


@pytest.mark.parametrize("kw", [k for k, _ in APPEND], ids=_name)
@pytest.mark.parametrize("rows_out", [True, False])
def test_append_in_4_bits(kw, rows_out):
    A.test_mxfp4(kw, rows_out)


@pytest.mark.parametrize("kw", [k for k, _ in APPEND], ids=_name)
@pytest.mark.parametrize("layout", ["heads first", "tokens first"])
def test_append_rows(kw, layout):
    A.test_row_type(kw, layout)

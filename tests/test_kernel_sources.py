"""Rules that the kernels' sources keep, checked on their text."""

import glob
import os
import re

import layerwise_qk_norm_qknorm_amd as qk

CSRC = os.path.join(os.path.dirname(os.path.abspath(qk.__file__)), "csrc")


def _code(path):
    """The file without comments."""
    text = open(path).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def test_inline_asm_holds_no_instructions():
    """The compiler puts the wait states that a matrix product's result needs before the
    instructions it knows that read it, and none before what stands in inline asm: an asm that
    reads such a register can get the value of before the product. So asm statements are empty
    (they only hide values from the optimizer)."""
    found = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*"))):
        for m in re.finditer(r"\basm\b\s*(?:volatile\s*)?\(\s*((?:\"[^\"]*\"\s*)+)", _code(path)):
            found += 1
            template = "".join(re.findall(r"\"([^\"]*)\"", m.group(1)))
            assert template.strip() == "", f"{os.path.basename(path)}: asm(\"{template}\" ...)"
    assert found > 5

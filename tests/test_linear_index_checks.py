"""The checked build's index checks in the products with activation, residual and experts, read from their sources: every
load or store of global memory whose address the kernels compute (the tensor copies do not count: their maps bound them)
stands in a statement that tests it first."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "block_scaled_precision_bsq_gb300", "csrc")
# what each source reads or writes, by the expressions that address it
ACCESSES = {
    "bsq_linear.cuh": [r"\boffsets\[", r"\bcounts\[", r"\bbias\[at\]", r"\bsums\[", r"reinterpret_cast<uint4\*>\(to\b"],
    "bsq_linear.cu": [r"\boffsets\[", r"\bown\["],
}


def source(name):
    with open(os.path.join(CSRC, name), encoding="utf-8") as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", " ", f.read(), flags=re.S)


def statement(code, at):
    """The statement around a place: to the next end and back to the last, past those inside parentheses."""
    depth, start = 0, at
    while start > 0:
        c = code[start - 1]
        depth += (c == ")") - (c == "(")
        if c in "{}" or c == ";" and depth == 0:
            break
        start -= 1
    return code[start:code.index(";", at)]


@pytest.mark.parametrize("name,pattern", [(n, p) for n, ps in ACCESSES.items() for p in ps])
def test_an_access_is_tested_first(name, pattern):
    code = source(name)
    found = [statement(code, m.start()) for m in re.finditer(pattern, code)]
    assert found
    for s in found:
        assert "in_bounds(" in s, "%s: %s" % (name, " ".join(s.split()))


def test_residuals_and_kept_arguments_are_tested_first():
    code = source("bsq_linear.cuh")
    copies = [statement(code, m.start()) for m in re.finditer(r"\bcopy_16\(to\b", code)]
    assert len(copies) == 1 and "there ? from" in copies[0] and "there ? 16 : 0" in copies[0]
    m = re.search(r"const bool there\b", code)
    assert "in_bounds(" in statement(code, m.start()) and "aux_len" in statement(code, m.start())
    assert len(re.findall(r"\baux \+", code)) == 1  # and nothing else reads them


def test_bias_gradients_are_tested_first():
    code = source("bsq_linear.cu")
    at = code.index("dbias[static_cast")
    guard = code.rfind("if (", 0, at)
    assert "in_bounds(" in code[guard:code.index("{", guard)] and code.count("dbias[") == 1

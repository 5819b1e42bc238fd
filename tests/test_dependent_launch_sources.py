"""Kernels that are launched with programmatic dependent launch are alive while the kernel before
still writes: what they read must come by ordinary loads, issued after the wait.  The non-coherent
path (__ldg, ld.global.nc, or const __restrict__ pointers, of which the compiler makes the same) is
for data that nothing writes during the kernel's life: here the weights of the GEMM alone."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "fp8_mxfp4_grouped_gb300", "csrc")
WEIGHTS = {"gemm.cu": {"w_scale"}}


def _code(path):
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", open(path).read(), flags=re.S)


def _dependent():
    return [p for p in sorted(glob.glob(os.path.join(CSRC, "*.cu")))
            if re.search(r"\b(start_dependent|griddep_wait)\(", _code(p))]


def test_the_files_are_found():
    names = {os.path.basename(p) for p in _dependent()}
    assert {"gemm.cu", "matvec.cu", "router.cu", "swiglu.cu", "tokens.cu"} <= names


@pytest.mark.parametrize("path", _dependent(), ids=os.path.basename)
def test_inputs_come_by_ordinary_loads(path):
    code, name = _code(path), os.path.basename(path)
    restricted = set(re.findall(r"\bconst\s+\w+\s*\*\s*__restrict__\s+(\w+)", code))
    assert restricted <= WEIGHTS.get(name, set())
    assert "ld.global.nc" not in code
    # the GEMM's one use is the wrapper that reads weight scales
    assert len(re.findall(r"\b__ldg\(", code)) == (1 if name in WEIGHTS else 0)
    if name in WEIGHTS:
        for call in re.findall(r"\bldg_u32\(([^;]*)", code):
            assert call.startswith(("wsrc", "const uint8_t* p")), call

"""The conversions and copies that the layer's operators share: each is called by something, and the
rule of the activations' scale stands once."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "fp8_mxfp4_grouped_gb300", "csrc")


def _code(path):
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", open(path).read(), flags=re.S)


ALL = "\n".join(_code(p) for p in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))))
COPIES = re.compile(r"^cp_async|^bulk_load$|^load$|ldmatrix|e2m1|e8m0|mma_f16|f32x2")
DEFINED = sorted({name for header in ("numeric.cuh", "ptx.cuh")
                  for name in re.findall(r"__device__ __forceinline__ [\w:<>\s*&]+?\b(\w+)\(",
                                         _code(os.path.join(CSRC, header)))
                  if header == "numeric.cuh" or COPIES.search(name)})


def test_functions_are_found():
    assert {"load", "quantize_codes", "e8m0_scale_code", "cp_async_16"} <= set(DEFINED)


@pytest.mark.parametrize("name", DEFINED)
def test_function_is_called(name):
    definitions = len(re.findall(r"__device__ __forceinline__ [\w:<>\s*&]+?\b%s\(" % name, ALL))
    assert len(re.findall(r"\b%s\(" % name, ALL)) > definitions


def test_one_rule_for_the_scale():
    # 448 * 2^e: the mantissa of 1.75, in either form, marks the rule
    assert len(re.findall(r"0x1FFFFFu|0x600000u", ALL)) == 1

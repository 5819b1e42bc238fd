"""Refusals at the limits of the MoE layer's entry points, before any CUDA call (no GPU needed)."""
import ctypes

import pytest

from tests.test_abi_moe_layer import BAD, OK, SHAPE, lib  # noqa: F401  (the fixture)


def _p(*addresses):
    return [ctypes.c_void_p(a) for a in addresses]


@pytest.mark.parametrize("rows,F,want", [(2 ** 31 - 1, 256, SHAPE), (2 ** 31 - 1, 128, SHAPE),
                                         (2 ** 24, 128 * 128, SHAPE), (1, 2 ** 31 - 128, BAD)])
def test_swiglu_sizes(lib, rows, F, want):  # noqa: F811
    # BAD is the missing pointer behind sizes that pass
    fwd = lib.lib.hg_swiglu_quantize(*_p(0x1000), rows, F, *_p(0x2000, 0, 0x4000, 0x5000), None)
    bwd = lib.lib.hg_swiglu_bwd(*_p(0x1000, 0x2000, 0), rows, F, *_p(0x4000), None)
    assert (fwd, bwd) == (want, want)
    assert lib.lib.hg_swiglu_quantize(*_p(0), 0, 128, *_p(0, 0, 0, 0), None) == OK

"""Waits in kernels: each is one of two forms, and the one that lets copies in flight land before a
CTA gives its memory back does not go by the caller's limit (hg_set_wait_timeout_us takes one
microsecond, less than a copy needs)."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "fp8_mxfp4_grouped_gb300", "csrc")


def _code(path):
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", open(path).read(), flags=re.S)


def _body(code, name):
    at = code.index("{", re.search(r"\b%s\(" % name, code).end())
    depth, i = 1, at + 1
    while depth:
        depth += {"{": 1, "}": -1}.get(code[i], 0)
        i += 1
    return code[at:i]


def test_draining_does_not_go_by_the_callers_limit():
    code = _code(os.path.join(CSRC, "hg_internal.cuh"))
    assert "timeout_ns" in _body(code, "wait_bounded")
    drain = _body(code, "wait_drain")
    assert "timeout_ns" not in drain and "abort" not in drain and "kDrainNs" in drain
    assert int(re.search(r"kDrainNs = (\d+)ull", code).group(1)) >= 10 ** 9


def test_no_other_wait_polls_a_barrier():
    for path in glob.glob(os.path.join(CSRC, "*.cu")):
        assert "mbar_try_wait" not in _code(path), path


def test_nothing_is_asked_for_after_giving_up():
    # between two runs of units the whole block agrees whether to go on, before
    # new rows are asked for on a barrier whose phase may never end
    code = _code(os.path.join(CSRC, "matvec.cu"))
    loop = code[code.index("for (int run = u0"):]
    assert loop.index("__syncthreads_or") < loop.index("load_run(")
    assert re.search(r"if \(__syncthreads_or\([^;]*abort[^;]*\)\) break;", loop)

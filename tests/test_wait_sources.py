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
    # input rows are asked for on a barrier with one arrival: not again in a phase
    # whose end the asking warp has not seen
    code = _code(os.path.join(CSRC, "matvec.cu"))
    ask = code[code.index("auto load_rows"):code.index("ptx::mbar_arrive_expect_tx(x_bar")]
    assert re.search(r"if \([^;]*!rows_came\) return;", ask)
    assert re.search(r"rows_came = __any_sync\([^;]*wait_bounded\(x_bar", code)
    assert re.search(r"warp == 0\) wait_drain\(x_bar, x_asked\)", code)

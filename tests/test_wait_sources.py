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


def test_draining_goes_on_until_a_limit_has_passed():
    # copies behind one that has landed may still be in flight: a loop over several drains ends
    # early only by a drain that has waited for its whole limit, never by the abort flag
    drain = _body(_code(os.path.join(CSRC, "hg_internal.cuh")), "wait_drain")
    assert re.search(r"> kDrainNs\) return false;\s*}\s*return true;", drain)
    loops = 0
    for path in glob.glob(os.path.join(CSRC, "*.cu")):
        code = _code(path)
        for drained in re.finditer(r"\bwait_drain\(", code):
            lines = code[:drained.start()].split("\n")
            if not any(re.search(r"\bfor \(", x) for x in lines[-4:]):
                continue
            loops += 1
            rest = code[drained.start():]
            after = rest[rest.index(";") + 1:][:80].strip()
            assert not re.match(r"if \([^;]*abort", after), path
            if re.match(r"[^;]*break;", rest):
                assert lines[-1].strip() == "if (!", path
    assert loops >= 5


def test_weight_gradient_waits_for_arrivals_after_giving_up():
    # the issuer's commits arrive on both CTAs: the odd one, which does not see the issuer's own
    # barrier, stays until the accumulators that it no longer waits for have been handed over
    code = _code(os.path.join(CSRC, "wgrad.cu"))
    epilogue = code[code.index("kRoleEpilogue"):code.index("bulk_wait_group_all")]
    assert re.search(r"!ok && i < 2; \+\+i\)\s*if \(!wait_drain\(bar_tfull \+ 8 \* \(\(tc \+ i\) & 1u\), "
                     r"\(\(tc \+ i\) >> 1\) & 1u\)\) break;", epilogue)

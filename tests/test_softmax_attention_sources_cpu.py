"""Rules that the tensor-core attention kernels keep and no run can show: read from their sources, no GPU is used."""
import os
import re

import pytest

import gated_linear_attention_local_b200 as sg

CSRC = os.path.join(os.path.dirname(os.path.abspath(sg.__file__)), "csrc")


def kernels():
    """{name: body} of the kernels whose warps split into roles."""
    out = {}
    for name in ("softmax_attn_fwd_tc.cu", "softmax_attn_bwd_tc.cu"):
        with open(os.path.join(CSRC, name)) as f:
            src = re.sub(r"//[^\n]*", "", f.read())
        for m in re.finditer(r"^(attn_\w+_kernel)\(.*?^\}", src, re.S | re.M):
            out[m.group(1)] = m.group(0)
    return out


KERNELS = kernels()


def test_the_three_kernels_are_found():
    assert set(KERNELS) == {"attn_fwd_tc_kernel", "attn_dkdv_tc_kernel", "attn_dq_tc_kernel"}


@pytest.mark.parametrize("name", sorted(KERNELS))
def test_registers_move_for_whole_warpgroups(name):
    """setmaxnreg is .aligned: all warps of a warpgroup execute one and the same instruction.  So there is one for the
    row warps (0 to 7) and one for the others (8 to 11), each ahead of any branch on the warp's role."""
    body = KERNELS[name]
    assert len(re.findall(r"setmaxnreg_dec<", body)) == 1 and len(re.findall(r"setmaxnreg_inc<", body)) == 1
    assert re.search(r"if \(warp >= 8\) \{\s*setmaxnreg_dec<", body)
    dec, inc = body.index("setmaxnreg_dec<"), body.index("setmaxnreg_inc<")
    assert re.search(r"\} else \{\s*$", body[:inc])
    # the branch that the dec opens is closed by the one that the inc follows
    between = body[body.rindex("if (warp >= 8) {", 0, dec):inc]
    depth = 0
    for i, c in enumerate(between):
        depth += (c == "{") - (c == "}")
        if depth == 0 and c == "}":
            assert re.fullmatch(r"\} else \{\s*", between[i:])
            break
    else:
        raise AssertionError("the two branches do not meet")


@pytest.mark.parametrize("name", sorted(KERNELS))
def test_no_wait_sends_lanes_different_ways(name):
    """A bounded wait can end differently in the lanes of a warp, and a lane that left a loop on its own answer would
    leave others at a warp-wide instruction.  So the warp votes (all_wait), or the answer is dropped (the abort flag
    says it to the item's end), or it only turns the lane's later waits off."""
    uses = re.findall(r"[^;{}]*[;{}]?[^;{}]*\bmbar_wait\(", KERNELS[name])
    assert uses
    for use in uses:
        assert re.search(r"(ok = ok && |auto wait = \[&\]\([^)]*\) \{ )mbar_wait\($", use), use.strip()
    assert re.search(r"auto wait = \[&\]\([^)]*\) \{ (return all_wait|mbar_wait)\(", KERNELS[name])

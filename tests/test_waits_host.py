"""Waits of the tensor-core kernels, by their source: each lane has a time limit of its own, so a role that goes on
with instructions of a whole warp (tcgen05.ld, shuffles, __syncwarp) must leave its loop with all lanes or none.
A limit that runs out cannot be brought about on a GPU without a kernel that is broken on purpose."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gemm_rocmfp2_mul_gb300", "csrc")
WAIT = r"\b(wait_for|mbar_wait)\("
VOTE = r"(goes_on\(|__all_sync\(0xffffffffu, |__any_sync\(0xffffffffu, )"


def alone(text):
    """The statements in which lanes of a whole warp wait and no vote follows."""
    role, found = "", []
    parts = [" ".join(p.split()) for p in re.split(r"(?<=[;{}])", re.sub(r"//[^\n]*", "", text))]
    for i, part in enumerate(parts):
        new_role = re.search(r"if \(((warp|lane)[^{]*)\) \{$", part)
        if new_role:
            role = new_role.group(1)
        if not re.search(WAIT, part) or "RFP2_DEV" in part or part.startswith("return"):
            continue
        if "lane == 0" in role or re.search(r"goes_on\(", part):
            continue
        # a value that this statement or one of the next hands to a vote
        name = re.search(r"(\w+) = [^;]*;$", part)
        if not (name and any(re.search(VOTE + name.group(1) + r"[,)]", p) for p in parts[i: i + 40])):
            found.append((role, part))
    return found


@pytest.mark.parametrize("name,waits", [("moe_gemm.cu", 9), ("gemm.cu", 9), ("nvfp4.cu", 8), ("verify.cu", 9)])
def test_lanes_leave_together(name, waits):
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    assert len(re.findall(WAIT, text)) >= waits
    assert alone(text) == []


def test_the_vote():
    with open(os.path.join(CSRC, "common.cuh")) as f:
        text = f.read()
    assert re.search(r"bool warp_goes_on\(bool there,[^{]*\{\s*if \(__all_sync\(0xffffffffu, there\)\) return true;", text)

"""Waits of the routed products' kernel, by its source: each lane has a time limit of its own, so a role that goes on
with instructions of a whole warp (tcgen05.ld, shuffles, __syncwarp) must leave its loop with all lanes or none.
A limit that runs out cannot be brought about on a GPU without a kernel that is broken on purpose."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gemm_rocmfp2_mul_gb300", "csrc")
WAIT = r"\b(wait_for|mbar_wait)\("


def alone(kernel):
    """The statements of a kernel's text in which lanes of a whole warp wait and no vote follows."""
    role, found = "", []
    parts = [" ".join(p.split()) for p in re.split(r"(?<=[;{}])", kernel)]
    for i, part in enumerate(parts):
        new_role = re.search(r"if \((warp[^{]*)\) \{$", part)
        if new_role:
            role = new_role.group(1)
        if not re.search(WAIT, part) or "lane == 0" in role or "goes_on(" in part:
            continue
        # a value that this statement or one of the next hands to a vote
        name = re.search(r"(\w+) = [^;]*;$", part)
        if not (name and any(re.search(rf"(goes_on\(|__all_sync\(0xffffffffu, ){name.group(1)}\)", p) for p in parts[i: i + 40])):
            found.append((role, part))
    return found


def test_lanes_leave_together():
    with open(os.path.join(CSRC, "moe_gemm.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    kernel = text[text.index("product_kernel(const __grid_constant__"): text.index("using ProductFn")]
    assert len(re.findall(WAIT, kernel)) >= 9
    assert alone(kernel) == []
    assert re.search(r"goes_on = \[&\]\(bool there\) \{\s*if \(__all_sync\(0xffffffffu, there\)\) return true;", kernel)

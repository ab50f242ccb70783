"""Checks of the serving side that need no GPU."""
import os
import re

from tests.test_abi import build_mod


def test_warps_that_share_a_barrier_leave_their_loop_together():
    """In a function with a barrier over several warps, no loop ends by a wait that each warp answers for itself: a warp
    that gave up would leave the others at the barrier."""
    seen = 0
    for name in ("attn_paged.cuh", "attn_paged_narrow.cuh"):
        text = re.sub(r"//[^\n]*", "", open(os.path.join(build_mod.CSRC, name)).read())
        for body in re.split(r"^(?=template|__device__|__global__)", text, flags=re.M):
            if "named_bar_sync(id" not in body:
                continue
            seen += 1
            loops = re.findall(r"while \((.*?)\) \{", body)
            assert loops and not any(re.search(r"\bwait\(|mbar_wait\(", x) for x in loops), loops
            assert any("wait_together(id" in x for x in loops)
    assert seen == 1  # the narrow form's softmax
    text = open(os.path.join(build_mod.CSRC, "attn_paged.cuh")).read()
    assert re.search(r"bool wait_together\(int id.*?\{\s*return named_bar_and\(id, 128, wait\(", text, flags=re.S)

"""Checks of the serving side that need no GPU."""
import ctypes
import os
import re

import pytest
import torch

from tests.test_abi import FAKE, build_mod
from tests.test_paged_abi import ints, lib, pool, rows, view  # noqa: F401  (lib: the fixture)

BF, I32 = torch.bfloat16, torch.int32


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


def test_guards_of_another_shape_or_type_are_refused(lib):  # noqa: F811
    import sequence_attn_fwd_gb300 as sa

    A = ctypes.addressof
    c, r = view(), rows()
    assert lib.paged_append_guarded(None, A(r), A(r), A(c), None, 0, 0, None, None, 9, 0, FAKE + 2, None) == 1
    assert lib.paged_reserve_guarded(FAKE, 8, FAKE, FAKE, FAKE, FAKE, FAKE + 1, 4, 8, 16, 16, None) == 1
    table, lens, refs = torch.zeros((2, 4), dtype=I32), torch.zeros(2, dtype=I32), torch.zeros(8, dtype=I32)
    for bad in (torch.zeros((4, 3), dtype=I32), torch.zeros((3, 2), dtype=I32), torch.zeros((4, 2)),
                torch.zeros((2, 4), dtype=I32).t()):
        with pytest.raises(ValueError, match="guard"):
            sa.paged_reserve(table, lens, refs, lens, 16, guard=bad)
    kp, x = torch.zeros((8, 1, 16, 64), dtype=BF), torch.zeros((1, 5, 64), dtype=BF)
    with pytest.raises(ValueError, match="CUDA"):  # the cache's tensors are looked at first
        sa.paged_append(x, x, kp, kp, table, lens, torch.zeros(3, dtype=I32), guard=torch.zeros((4, 3), dtype=I32))


def test_positions_for_a_cache_that_does_not_turn_are_refused():
    import sequence_attn_fwd_gb300 as sa

    cache = sa.PagedCache(4, 1, 64, rows=1, max_pages=4, device="cpu")
    x = torch.zeros((1, 1, 64), dtype=BF)
    with pytest.raises(ValueError, match="plan"):
        cache.step(0, x, x, x, torch.zeros(2, dtype=I32), torch.zeros((1, 1), dtype=I32))


def test_layers_are_counted_in_64_bits(lib):  # noqa: F811
    """Four pools of 2^30 layers are refused, not taken for none at all."""
    pools = pool(4, n_layers=1 << 30)
    s, d = ints(0), ints(1)
    A = ctypes.addressof
    assert lib.paged_copy(A(pools), 4, A(s), A(d), 1, 16, None) == 2
    pools = pool(2, n_layers=(1 << 31) - 1)
    assert lib.paged_copy(A(pools), 2, A(s), A(d), 1, 16, None) == 2
    big = (1 << 63) - 16  # bytes of a page, which rounded up to whole copies would pass 64 bits
    assert lib.paged_copy(A(pool(page_bytes=big, page_stride=big)), 1, A(s), A(d), 1, 16, None) == 2


def test_strides_of_pool_dimensions_of_one_are_free():
    """One KV head: its stride may be anything, in either pool. (Past the layout checks, the refusal is that of CPU tensors.)"""
    import sequence_attn_fwd_gb300 as sa

    kp = torch.zeros((8, 1, 16, 64), dtype=BF)
    vp = torch.zeros((8, 16, 1, 64), dtype=BF).transpose(1, 2)
    assert vp.shape == kp.shape and vp.stride() != kp.stride()
    q = torch.zeros((4, 2, 64), dtype=BF)
    table, lens, cu = torch.zeros((1, 4), dtype=I32), torch.zeros(1, dtype=I32), torch.zeros(2, dtype=I32)
    for a, b in ((kp, vp), (vp, kp)):
        with pytest.raises(ValueError, match="CUDA"):
            sa.attn_paged(q, a, b, table, lens, cu)
    both = torch.zeros((8, 2, 16, 64), dtype=BF)
    with pytest.raises(ValueError, match="pools"):
        sa.attn_paged(q, both, torch.zeros((8, 16, 2, 64), dtype=BF).transpose(1, 2), table, lens, cu)

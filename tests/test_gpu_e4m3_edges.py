"""The 8-bit cache where its kernels hand work from one warpgroup to the other."""
import pytest
import torch

from tests.test_gpu_drafts import Cache, queries, sa  # noqa: F401
from tests.test_gpu_paged import i32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,G,q_len", [(128, 1, 1), (128, 4, 3), (64, 16, 1), (64, 2, 8)])
def test_items_joined_by_one_warpgroup_for_both(sa, D, G, q_len):  # noqa: F811
    """Up to 16 rows: one warpgroup reads what the other's products left, item behind item of two to five tiles (odd and even
    numbers of them, so that either warpgroup has the first and the last one)."""
    B = 1200
    kv = [129 + (b * 71) % 512 for b in range(B)]
    c = Cache([q_len] * B, kv, 2, D, 16, True, 3)
    q = queries(q_len * B, 2 * G, D)
    first = sa.attn_paged(q, *c.args(), **c.kw)
    for _ in range(20):
        again = sa.attn_paged(q, *c.args(), **c.kw)
        assert torch.equal(again[0], first[0]) and torch.equal(again[1], first[1])
    few = list(range(0, B, 97))
    pick = torch.cat([torch.arange(b * q_len, (b + 1) * q_len) for b in few]).cuda()
    c.table, c.lens, c.cu = c.table[few], c.lens[few], i32([i * q_len for i in range(len(few) + 1)])
    c.check((first[0][:, pick], first[1][:, pick]), q[:, pick])

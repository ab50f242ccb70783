"""The serving side where something is not there: missing pages in front of very low scores, rows without room,
forks of evicted pages, pairs that are not turned."""
import math

import pytest
import torch

from tests import paged_ref as ref
from tests.test_gpu_paged import i32, make_cache

pytestmark = pytest.mark.gpu
BF, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module")
def sa(cuda_dev):
    import sequence_attn_fwd_gb300 as sa

    yield sa
    sa.query_device_error()


# ---------------------------------------------------------------------------- missing pages, low scores
def low_scores(new, kv, Hq, Hkv, D, ps, seed):
    """A cache and queries whose scores all lie near -16 sqrt(D): -128 with heads of 64, -181 with 128."""
    kp, vp, table, lens, cu = make_cache(new, kv, Hkv, D, ps, seed)
    kp.copy_(torch.where(kp.isnan(), kp, kp * 0.25 - 4.0))
    g = torch.Generator().manual_seed(seed + 1)
    q = (torch.randn((Hq, sum(new), D), generator=g) * 0.25 + 4.0).to(BF).cuda()
    return q, kp, vp, table, lens, cu


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ps", [16, 256])
@pytest.mark.parametrize("causal", [True, False])
def test_low_scores_behind_missing_first_pages(sa, D, ps, causal):
    """More items than CTAs, so that some are whole: the first 256 of 640 keys are not there."""
    new, kv = [33 + b % 7 for b in range(120)], [640 - b % 5 for b in range(120)]
    q, kp, vp, table, lens, cu = low_scores(new, kv, 4, 2, D, ps, D + ps)
    table[:, :256 // ps] = -1
    got = sa.attn_paged(q, kp, vp, table, lens, cu, causal=causal)
    ref.check_attention(got, ref.attention(q, kp, vp, table, lens, cu, causal, 1 / math.sqrt(D)))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("hole", [(0, 20000), (10000, 40000), (59000, 60000)])
def test_low_scores_behind_a_missing_stretch_of_a_cut_item(sa, D, hole):
    """One long sequence over all CTAs: ranges begin inside the missing stretch and end behind it."""
    ps = 16
    q, kp, vp, table, lens, cu = low_scores([70], [60000], 2, 2, D, ps, D + hole[0])
    table[0, hole[0] // ps:hole[1] // ps] = -1
    got = sa.attn_paged(q, kp, vp, table, lens, cu)
    ref.check_attention(got, ref.attention(q, kp, vp, table, lens, cu, True, 1 / math.sqrt(D)))


def test_low_scores_behind_missing_pages_few_rows(sa):
    """The same for single tokens and drafts."""
    q, kp, vp, table, lens, cu = low_scores([1, 6, 1], [3000, 700, 40000], 8, 2, 128, 16, 5)
    table[0, :100], table[1, :20], table[2, 500:2000] = -1, -1, -1
    got = sa.attn_paged(q, kp, vp, table, lens, cu)
    ref.check_attention(got, ref.attention(q, kp, vp, table, lens, cu, True, 1 / math.sqrt(128)))

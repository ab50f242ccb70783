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


# ---------------------------------------------------------------------------- rows without room
def filled_cache(sa, rows=4, n_pages=10, seed=1):
    """Rows 0 and 1 hold 48 and 20 tokens (16 a page), row 2 is a fork of row 0 (every page shared); 5 pages are free."""
    cache = sa.PagedCache(n_pages, 2, 64, rows=rows, max_pages=9, page_size=16, layers=2, plan=sa.RopePlan(64, (32,)))
    for p in (cache.k_pages, cache.v_pages):
        p.copy_(torch.randn(p.shape, generator=torch.Generator().manual_seed(seed)).to(BF))
    assert cache.reserve(i32([48, 20] + [0] * (rows - 2))).tolist() == [0] * rows
    assert cache.fork([0], [2]).tolist() == [0]
    return cache


def tokens(total, seed=2):
    g = torch.Generator().manual_seed(seed)
    q, k, v = (torch.randn((H, total, 64), generator=g).to(BF).cuda() for H in (4, 2, 2))
    return q, k, v, torch.arange(total, dtype=I32, device="cuda")[None] + 60


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("n_new,why", [([200, 2, 1, 0], 2), ([96, 2, 1, 0], 1)])
def test_a_row_without_room_keeps_its_keys(sa, n_new, why, captured):
    """Row 0's request is refused (its table is too short, or the pool): its tokens are dropped and see nothing, the
    keys that it and its fork hold stay as they are, and the rows that got room are served as if it were not there."""
    cache, other = filled_cache(sa), filled_cache(sa)
    cu = i32([0] + torch.tensor(n_new).cumsum(0).tolist())
    q, k, v, pos = tokens(sum(n_new))
    before = cache.k_pages.clone(), cache.v_pages.clone()
    held = cache.page_table[0, :3].long()
    n = i32(n_new)

    def step(c, n, q, k, v, cu, pos):
        """Both layers; each twice, as the second time writes what the first one wrote."""
        status = c.reserve(n)
        for layer in (0, 1, 0, 1):
            o = c.step(layer, q, k, v, cu, pos)
        return status, o

    if captured:
        warm = filled_cache(sa)
        step(warm, n, q, k, v, cu, pos)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            status, (o, lse) = step(cache, n, q, k, v, cu, pos)
        graph.replay()
    else:
        status, (o, lse) = step(cache, n, q, k, v, cu, pos)
    got = status.tolist()
    assert got[0] == why
    for pool, old in zip((cache.k_pages, cache.v_pages), before):
        assert torch.equal(pool[:, held], old[:, held])
    a = n_new[0]
    assert (o[:, :a] == 0).all() and torch.isneginf(lse[:, :a]).all()
    # the same step without row 0's request, and without the rows that were refused with it
    served = [0] + [m if s == 0 else 0 for m, s in zip(n_new[1:], got[1:])]
    if why == 2:
        assert served[1:] == n_new[1:]
    keep = torch.cat([torch.arange(int(cu[b]), int(cu[b + 1])) for b in range(4) if served[b]] or [torch.zeros(0).long()])
    if len(keep):
        _, (wo, wl) = step(other, i32(served), *(t[:, keep].contiguous() for t in (q, k, v)),
                           i32([0] + torch.tensor(served).cumsum(0).tolist()), pos[:, keep].contiguous())
        assert torch.equal(o[:, keep], wo) and torch.equal(lse[:, keep], wl)
        assert torch.equal(cache.k_pages, other.k_pages) and torch.equal(cache.v_pages, other.v_pages)
    # a request that fits, afterwards, is served
    n2 = i32([1, 0, 0, 0])
    status, (o, lse) = step(cache, n2, q[:, :1], k[:, :1], v[:, :1], i32([0, 1, 1, 1, 1]), pos[:, :1])
    assert status.tolist() == [0] * 4 and torch.isfinite(lse).all()
    assert torch.equal(cache.v_pages[1, int(cache.page_table[0, 3]), :, 0], v[:, 0])


def test_reserve_results_stay_apart_and_rows_may_change_between_steps(sa):
    """Each reserve's answer is a tensor of its own; a table changed through the functions is served by the cache."""
    cache = filled_cache(sa)
    first = cache.reserve(i32([200, 1, 0, 0]))
    second = cache.reserve(i32([0, 0, 0, 3]))
    assert first.tolist() == [2, 0, 0, 0] and second.tolist() == [0] * 4
    own = sa.PagedCache(12, 2, 64, rows=1, max_pages=9)
    assert sa.paged_reserve(own.page_table, own.kv_lens, own.page_refs, i32([5]), 16).tolist() == [0]
    q, k, v, _ = tokens(5)
    o, lse = own.step(0, q, k, v, i32([0, 5]))
    assert torch.isfinite(lse).all() and torch.equal(own.k_pages[0, 0, :, :5], k)


def test_requests_between_two_steps(sa):
    """A row that was granted tokens and refused more brings the granted ones; one that brings all keeps its keys."""
    q, k, v, pos = tokens(60)
    for bring, ok in ((3, True), (60, False)):
        cache = filled_cache(sa)
        held = cache.page_table[0, :3].long()
        before = cache.k_pages[0, held].clone()
        assert cache.reserve(i32([3, 0, 0, 0])).tolist() == [0] * 4
        assert cache.reserve(i32([0, 0, 1, 0])).tolist() == [0] * 4  # another row's request in between
        assert cache.reserve(i32([200, 0, 0, 0])).tolist() == [2, 0, 0, 0]
        assert cache.reserve(i32([0, 2, 0, 0])).tolist() == [0] * 4
        o, lse = cache.step(0, q[:, :bring], k[:, :bring], v[:, :bring], i32([0] + [bring] * 4), pos[:, :bring])
        assert torch.equal(cache.k_pages[0, held], before)
        assert torch.isfinite(lse).all() if ok else (torch.isneginf(lse).all() and (o == 0).all())


def test_a_refused_row_starts_over(sa):
    """Freed, forked into or asked again with success, a row is served as any other."""
    q, k, v, pos = tokens(9)
    cache = filled_cache(sa)
    assert cache.reserve(i32([200, 0, 200, 0])).tolist() == [2, 0, 2, 0]
    cache.free([0, 2])
    assert cache.fork([1], [2]).tolist() == [0]
    assert cache.reserve(i32([9, 0, 0, 0])).tolist() == [0] * 4  # shorter than it was when it was refused
    o, lse = cache.step(0, q, k, v, i32([0, 9, 9, 9, 9]), pos)
    assert torch.isfinite(lse).all() and torch.equal(cache.v_pages[0, int(cache.page_table[0, 0]), :, :9], v)
    assert cache.reserve(i32([0, 0, 9, 0])).tolist() == [0] * 4
    o, lse = cache.step(0, q, k, v, i32([0, 0, 0, 9, 9]), pos)
    assert torch.isfinite(lse).all() and cache.kv_lens.tolist() == [9, 20, 29, 0]
    assert cache.reserve(i32([0, 0, 200, 0])).tolist() == [0, 0, 2, 0]
    assert cache.reserve(i32([0, 0, 2, 0])).tolist() == [0] * 4
    o, lse = cache.step(0, q[:, :2], k[:, :2], v[:, :2], i32([0, 0, 0, 2, 2]), pos[:, :2])
    assert torch.isfinite(lse).all() and cache.kv_lens[2] == 31


def test_guarded_calls_of_a_caller_without_the_handle(sa):
    """The functions on tensors of the caller's own, and without a guard the plain calls."""
    cache = filled_cache(sa)
    guard = torch.zeros((4, 4), dtype=I32, device="cuda")
    t, pools = (cache.page_table, cache.kv_lens), (cache.k_pages[0], cache.v_pages[0])
    q, k, v, _ = tokens(8)
    before = cache.k_pages.clone()
    cu = i32([0, 4, 8, 8, 8])
    assert sa.paged_reserve(*t, cache.page_refs, i32([200, 4, 0, 0]), 16, guard=guard).tolist() == [2, 0, 0, 0]
    sa.paged_append(k, v, *pools, *t, cu, guard=guard)
    o, lse = sa.attn_paged(q, *pools, cache.page_table, guard[3], cu)
    assert torch.isneginf(lse[:, :4]).all() and torch.isfinite(lse[:, 4:]).all()
    assert torch.equal(cache.k_pages[:, cache.page_table[0, :3].long()], before[:, cache.page_table[0, :3].long()])
    _, plain = sa.attn_paged(q, *pools, *t, cu)
    assert torch.isfinite(plain).all() and torch.equal(plain[:, 4:], lse[:, 4:])


# ---------------------------------------------------------------------------- forks of evicted pages
@pytest.mark.parametrize("entry", [-1, 10 ** 6])
def test_fork_of_a_row_whose_last_page_was_evicted(sa, entry):
    """The child holds what its parent holds: no page where the parent has none, and none is taken from the pool."""
    cache = filled_cache(sa)
    cache.k_pages.fill_(math.nan)  # what a page that no one has written may hold
    cache.v_pages.fill_(math.inf)
    gone = int(cache.page_table[1, 1])
    cache.page_table[1, 1] = entry  # the partly filled last page of row 1, given up by the caller
    cache.page_refs[gone] -= 1
    live = cache.page_refs.clone()
    first = int(cache.page_table[1, 0])
    g = torch.Generator().manual_seed(3)
    for p in (cache.k_pages, cache.v_pages):
        p[:, first] = torch.randn(p[:, first].shape, generator=g).to(BF).cuda()
    assert cache.fork([1, 0], [3, 2]).tolist() == [0, 3]
    assert cache.page_table[3].tolist() == [first, entry] + [-1] * 7 and cache.kv_lens[3] == 20
    live[first] += 1
    assert torch.equal(cache.page_refs, live)
    assert cache.kv_lens.tolist() == [48, 20, 48, 20]
    q = torch.randn((4, 1, 64), generator=g).to(BF).cuda()
    see = [sa.attn_paged(q, cache.k_pages[0], cache.v_pages[0], cache.page_table, cache.kv_lens, i32(cu), causal=False)
           for cu in ([0, 0, 1, 1, 1], [0, 0, 0, 0, 1])]  # the parent's row, the child's
    assert torch.isfinite(see[0][1]).all()
    assert torch.equal(see[0][0], see[1][0]) and torch.equal(see[0][1], see[1][1])


def test_forks_of_evicted_and_of_whole_rows_in_one_call(sa):
    """Rows that end in a page, at its end, in an evicted page, and in a table's last column."""
    ps, W = 16, 4
    table = i32([[0, 1, 2, 3], [4, 5, -1, -1], [6, -1, 8, -1], [9, -1, -1, -1]] + [[-1] * W] * 5)
    lens = i32([64, 23, 45, 21, 0, 0, 0, 0, 0])  # row 3 ends in column 1, evicted; row 2 lost its middle
    refs = torch.zeros(16, dtype=I32, device="cuda")
    refs[[0, 1, 2, 3, 4, 5, 6, 8, 9]] = 1
    pool = torch.arange(16.0, device="cuda")[:, None, None, None].expand(16, 1, ps, 64).contiguous()
    status = sa.paged_fork(pool, table, lens, refs, [3, 1, 2, 0, 1], [4, 5, 6, 7, 8])
    assert status.tolist() == [0] * 5 and lens.tolist() == [64, 23, 45, 21, 21, 23, 45, 64, 23]
    assert table[4:].tolist() == [[9, -1, -1, -1], [4, 7, -1, -1], [6, -1, 10, -1], [0, 1, 2, 3], [4, 11, -1, -1]]
    assert refs.tolist() == [2, 2, 2, 2, 3, 1, 2, 1, 1, 2, 1, 1, 0, 0, 0, 0]
    assert [pool[p].unique().tolist() for p in (7, 10, 11)] == [[5.0], [8.0], [5.0]]


# ---------------------------------------------------------------------------- pairs that are not turned
@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("S", [3, 6000])
def test_pairs_without_an_axis_are_copied(sa, dtype, interleaved, S):
    """Whatever they hold: infinities, NaN, signed zeros stay in their own elements."""
    D = 64
    plan = sa.RopePlan(D, (5, 6))  # eleven pairs turn, 21 do not
    x = torch.randn((1, 2, S, D), generator=torch.Generator().manual_seed(S)).to(dtype)
    first = torch.arange(11, 32) * 2 if interleaved else torch.arange(11, 32)
    second = first + 1 if interleaved else first + 32
    odd = torch.tensor([math.inf, -math.inf, math.nan, -0.0, 3e38])
    x[..., first[:20]] = odd.repeat(4).to(dtype)
    x[..., second[:20]] = odd.repeat_interleave(4).to(dtype)
    x = x.cuda()
    pos = torch.randint(0, 10 ** 6, (2, 1, S), generator=torch.Generator().manual_seed(1)).to(I32).cuda()
    still = torch.cat([first, second]).cuda()
    bits = torch.int16 if dtype == BF else torch.int32

    def copied(y, x):
        y, x = y[..., still], x[..., still]
        assert torch.equal(y.isnan(), x.isnan())
        assert torch.equal(y.view(bits)[~x.isnan()], x.view(bits)[~x.isnan()])

    for fn in (sa.rope_axes, sa.rope_axes_bwd):
        copied(fn(x, None, pos, *plan, interleaved=interleaved)[0], x)
    if dtype == BF:
        cache = sa.PagedCache(400, 2, D, rows=1, max_pages=400, plan=plan, interleaved=interleaved)
        assert cache.reserve(i32([S])).tolist() == [0]
        q = sa.paged_append(x[0], x[0], cache.k_pages[0], cache.v_pages[0], cache.page_table, cache.kv_lens, i32([0, S]),
                            q=x[0], positions=pos[:, 0], inv_freq=plan.inv_freq, axes=plan.axes, interleaved=interleaved)
        copied(q, x[0])
        copied(cache.k_pages[0].transpose(0, 1).reshape(2, -1, D)[:, :S], x[0])

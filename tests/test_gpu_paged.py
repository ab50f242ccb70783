"""The serving-side kernels against their 64-bit definitions (tests/paged_ref.py)."""
import math

import pytest
import torch

from tests import paged_ref as ref

pytestmark = pytest.mark.gpu
BF, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module")
def sa(cuda_dev):
    import sequence_attn_fwd_gb300 as sa

    yield sa
    sa.query_device_error()


def i32(x):
    return torch.tensor(x, dtype=I32, device="cuda")


def make_cache(new, kv, Hkv, D, ps, seed=0, extra_width=2, garbage=True, shared_pool=False):
    """Pools whose unused slots hold NaN and inf, a shuffled table, lengths and offsets."""
    g = torch.Generator().manual_seed(seed)
    pages = [-(-n // ps) for n in kv]
    n_pages = sum(pages) + 5
    ids = torch.randperm(n_pages, generator=g)
    table = torch.full((len(kv), max(pages + [1]) + extra_width), -1, dtype=I32)
    kp = torch.randn((n_pages, Hkv, ps, D), generator=g).to(BF)
    vp = torch.randn((n_pages, Hkv, ps, D), generator=g).to(BF)
    if garbage:
        used = torch.zeros((n_pages, ps), dtype=torch.bool)
    at = 0
    for b, n in enumerate(pages):
        table[b, :n] = ids[at:at + n].to(I32)
        at += n
        for i in range(n):
            if garbage:
                used[table[b, i], :max(0, min(ps, kv[b] - i * ps))] = True
    if garbage:
        bad = ~used[:, None, :, None].expand(n_pages, Hkv, ps, D)
        kp, vp = kp.masked_fill(bad, math.nan), vp.masked_fill(bad, math.inf)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    if shared_pool:  # K and V pages side by side in one allocation
        both = torch.stack([kp, vp], 1).cuda()
        kp, vp = both[:, 0], both[:, 1]
    return kp.cuda(), vp.cuda(), table.cuda(), i32(kv), i32(cu)


def run_case(sa, new, kv, Hq, Hkv, D, ps, causal, token_major=True, scale=None, seed=0, holes=(), behind=0, **kw):
    kp, vp, table, lens, cu = make_cache(new, kv, Hkv, D, ps, seed, **kw)
    for b, i, page in holes:
        table[b, i] = page
    total = sum(new) + behind
    g = torch.Generator().manual_seed(seed + 1)
    q = torch.randn((total, Hq, D) if token_major else (Hq, total, D), generator=g).to(BF).cuda()
    q = q.transpose(0, 1) if token_major else q
    out = torch.full((total, Hq, D), 7.0, dtype=BF, device="cuda").transpose(0, 1)
    lse = torch.full((Hq, total), 7.0, device="cuda")
    sa.attn_paged(q, kp, vp, table, lens, cu, causal=causal, scale=scale, out=out, lse=lse)
    r = ref.attention(q, kp, vp, table, lens, cu, causal, scale or 1 / math.sqrt(D))
    ref.check_attention((out, lse), r)
    if behind:
        assert (out[:, total - behind:] == 7).all() and (lse[:, total - behind:] == 7).all()
    return out, lse


@pytest.mark.parametrize("ps", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("D", [64, 128])
def test_page_sizes_and_ragged_ends(sa, ps, D):
    run_case(sa, [1, 3, 40], [1, 129, 300], 4, 2, D, ps, True, seed=ps + D)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (28, 4), (8, 1), (6, 2), (40, 1), (128, 1)])
@pytest.mark.parametrize("causal", [True, False])
def test_head_groups(sa, Hq, Hkv, causal):
    run_case(sa, [1, 19, 2], [517, 40, 128], Hq, Hkv, 128, 16, causal, token_major=Hq % 2 == 0, seed=Hq)


@pytest.mark.parametrize("new,kv", [
    ([1], [1]),
    ([1], [128]),
    ([1], [129]),
    ([1, 0, 1], [200, 64, 0]),      # a row without new tokens, a row without keys
    ([5], [3]),                      # more new tokens than keys: the first see none
    ([300], [120]),                  # whole tiles of rows that see none
    ([700, 1, 37], [700, 900, 37]),  # a prompt from its beginning, several row blocks
    ([0, 0], [10, 10]),
])
@pytest.mark.parametrize("causal", [True, False])
def test_lengths(sa, new, kv, causal):
    run_case(sa, new, kv, 14, 2, 64, 16, causal, seed=len(new) + kv[0], behind=3)


def test_many_short_sequences(sa):
    """More sequences than threads in a CTA, more CTAs than tiles in places."""
    new = [(b * 7) % 3 for b in range(600)]
    kv = [n + (b * 37) % 90 for b, n in enumerate(new)]
    run_case(sa, new, kv, 2, 1, 64, 16, True, seed=3)


def test_one_long_sequence_over_all_ctas(sa):
    run_case(sa, [2], [30011], 8, 2, 128, 64, True, seed=4)


def test_pages_that_are_missing(sa):
    """Table entries that are no page: those keys are not seen; a row that only has such pages sees nothing."""
    holes = [(0, 0, -1), (0, 3, 10 ** 9), (0, 8, -2 ** 31), (1, 0, -5), (2, 1, 2 ** 31 - 1)]
    run_case(sa, [9, 2, 33], [300, 14, 290], 4, 2, 128, 16, True, seed=5, holes=holes)
    run_case(sa, [9, 2], [700, 290], 4, 2, 64, 256, True, seed=6, holes=[(0, 1, -1), (1, 0, 99)])


def test_strides_and_pools_side_by_side(sa):
    for tm in (True, False):
        run_case(sa, [3, 50], [400, 77], 6, 2, 128, 32, True, token_major=tm, seed=7, shared_pool=True)


def test_large_scores_and_scale(sa):
    """Scores of a few hundred, and a key far above all others late in a row: the running reference moves."""
    new, kv = [3], [1000]
    kp, vp, table, lens, cu = make_cache(new, kv, 1, 128, 16, 11)
    q = (torch.randn((2, 3, 128)) * 6).to(BF).cuda()
    kp[table[0, 60].item(), 0, 5] = (q[0, 0].float() * 0.5).to(BF)
    for scale in (None, 0.5):
        got = sa.attn_paged(q, kp, vp, table, lens, cu, scale=scale)
        ref.check_attention(got, ref.attention(q, kp, vp, table, lens, cu, True, scale or 1 / math.sqrt(128)))


def test_lengths_beyond_the_table_and_broken_offsets_stay_inside(sa):
    """kv_lens past the table counts as the table; offsets past total are cut: nothing outside is touched."""
    kp, vp, table, lens, cu = make_cache([4, 4], [64, 64], 2, 64, 16, 12, extra_width=0)
    q = torch.randn((4, 8, 64)).to(BF).cuda()
    long = i32([1000, -7])
    got = sa.attn_paged(q, kp, vp, table, long, cu, causal=False)
    ref.check_attention(got, ref.attention(q, kp, vp, table, i32([64, 0]), cu, False, 1 / 8))
    guard = torch.full((4, 8 + 64, 64), 7.0, dtype=BF, device="cuda")
    sa.attn_paged(q, kp, vp, table, lens, i32([0, 4, 900]), out=guard[:, 32:40])
    sa.attn_paged(q, kp, vp, table, lens, i32([-3, 6, 2]), out=guard[:, 32:40])
    assert (guard[:, :32] == 7).all() and (guard[:, 40:] == 7).all()


def test_repeated_calls_are_bitwise_equal_and_streams(sa):
    kp, vp, table, lens, cu = make_cache([1] * 5 + [60], [3000, 17, 900, 128, 4001, 700], 2, 128, 16, 13)
    q = torch.randn((14, 65, 128)).to(BF).cuda()
    a = sa.attn_paged(q, kp, vp, table, lens, cu)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = sa.attn_paged(q, kp, vp, table, lens, cu)
    torch.cuda.current_stream().wait_stream(side)
    c = sa.attn_paged(q, kp, vp, table, lens, cu)
    for x in (b, c):
        assert torch.equal(a[0], x[0]) and torch.equal(a[1], x[1])


def test_captured_call_follows_lengths_and_tables(sa):
    """One captured call replayed on other lengths, tables and offsets equals a fresh call on them."""
    kp, vp, table, lens, cu = make_cache([1, 1, 2], [400, 33, 2000], 2, 128, 16, 14, garbage=False)
    q = torch.randn((6, 4, 128)).to(BF).cuda()
    ws = torch.empty(sa.attn_paged_workspace_bytes(6, 2, 4, 128), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(q), torch.empty((6, 4), device="cuda")
    sa.attn_paged(q, kp, vp, table, lens, cu, out=out, lse=lse, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sa.attn_paged(q, kp, vp, table, lens, cu, out=out, lse=lse, workspace=ws)
    for new_lens, new_cu, flip in (([400, 33, 2000], [0, 1, 2, 4], False), ([12, 500, 129], [0, 2, 2, 4], True)):
        lens.copy_(i32(new_lens))
        cu.copy_(i32(new_cu))
        if flip:
            table.copy_(table.flip(0))
            table.clamp_(min=0)
        graph.replay()
        torch.cuda.synchronize()
        fresh = sa.attn_paged(q, kp, vp, table, lens, cu)
        assert torch.equal(out, fresh[0]) and torch.equal(lse, fresh[1])
        ref.check_attention((out, lse), ref.attention(q, kp, vp, table, lens, cu, True, 1 / math.sqrt(128)))


def test_rows_behind_the_sequences_may_hold_anything(sa):
    """NaN and inf in query rows of no sequence reach no other row, in either form of the kernel."""
    for new, kv in (([1, 2], [300, 40]), ([70, 1], [300, 140])):
        kp, vp, table, lens, cu = make_cache(new, kv, 2, 128, 16, 15)
        q = torch.randn((8, sum(new) + 9, 128)).to(BF).cuda()
        q[:, sum(new):sum(new) + 4], q[:, sum(new) + 4:] = math.nan, math.inf
        out = torch.full_like(q, 7.0)
        got = sa.attn_paged(q, kp, vp, table, lens, cu, out=out)
        ref.check_attention(got, ref.attention(q, kp, vp, table, lens, cu, True, 1 / math.sqrt(128)))
        assert (out[:, sum(new):] == 7).all()


@pytest.mark.parametrize("new", [[1, 3, 1], [80, 3, 1]])
def test_a_nan_query_stays_nan(sa, new):
    """A row with a NaN score is NaN with a NaN lse, also when its keys were split; no other row is."""
    kp, vp, table, lens, cu = make_cache(new, [5000, 40, 20], 2, 128, 16, 20)
    q = torch.randn((2, sum(new), 128)).to(BF).cuda()
    bad = q.clone()
    bad[1, 0, 5] = math.nan
    want = sa.attn_paged(q, kp, vp, table, lens, cu)
    o, lse = sa.attn_paged(bad, kp, vp, table, lens, cu)
    assert o[1, 0].isnan().all() and lse[1, 0].isnan()
    want[0][1, 0], want[1][1, 0] = o[1, 0], lse[1, 0]
    assert torch.equal(o.nan_to_num(), want[0].nan_to_num()) and torch.equal(lse.nan_to_num(), want[1].nan_to_num())


def test_strides_of_dimensions_of_one_are_free(sa):
    kp, vp, table, lens, cu = make_cache([1], [77], 2, 64, 16, 22)
    q = torch.randn((4, 1, 64)).to(BF).cuda()
    want = sa.attn_paged(q, kp, vp, table, lens, cu)
    odd = q.as_strided((4, 1, 64), (64, 3, 1))
    out = torch.empty_like(q).as_strided((4, 1, 64), (64, 5, 1))
    got = sa.attn_paged(odd, kp, vp, table, lens, cu, out=out)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_no_pages_no_lse_and_a_table_without_columns(sa):
    kp, vp, table, lens, cu = make_cache([3, 1], [50, 20], 2, 64, 16, 16)
    q = torch.randn((4, 4, 64)).to(BF).cuda()
    none = torch.zeros((2, 0), dtype=I32, device="cuda")
    o, lse = sa.attn_paged(q, kp, vp, none, lens, cu)
    assert (o == 0).all() and torch.isneginf(lse).all()
    o, lse = sa.attn_paged(q, kp, vp, torch.full_like(table, -1), lens, cu)
    assert (o == 0).all() and torch.isneginf(lse).all()
    # the C call without lse gives the same O
    import ctypes

    from sequence_attn_fwd_gb300 import paged

    want = sa.attn_paged(q, kp, vp, table, lens, cu)[0]
    out, ws = torch.empty_like(q), torch.empty(sa.attn_paged_workspace_bytes(4, 2, 4, 64), dtype=torch.uint8, device="cuda")
    view = paged._cache_view(kp, vp, table, lens, cu)[0]
    assert sa.lib.attn_paged(q.data_ptr(), q.stride(0), q.stride(1), view, out.data_ptr(), q.stride(0), q.stride(1), None,
                             ws.data_ptr(), ws.numel(), 4, 4, 1, ctypes.c_float(1 / 8),
                             torch.cuda.current_stream().cuda_stream) == 0
    assert torch.equal(out, want)


def test_most_sequences_of_a_call(sa):
    B = 4096
    new = [1 if b % 3 else 0 for b in range(B)]
    kv = [n + b % 23 for b, n in enumerate(new)]
    run_case(sa, new, kv, 2, 2, 64, 16, True, seed=17)
    with pytest.raises(sa.AttnError):
        run_case(sa, new + [1], kv + [1], 2, 2, 64, 16, True, seed=17)


@pytest.mark.parametrize("new,kv", [([4] * 40, [257] * 40), ([8, 1, 8], [5000, 4000, 640]), ([64] * 3, [64, 200, 900]),
                                    ([2, 65], [700, 1300]), ([129, 128, 127], [140, 128, 1000])])
@pytest.mark.parametrize("G", [1, 7, 8])
def test_row_counts_around_the_tiles(sa, new, kv, G):
    """Rows per KV head below, at and above 16, 32, 64 and the tiles of 128; items that ranges cut anywhere."""
    run_case(sa, new, kv, 2 * G, 2, 128, 32, True, seed=G)
    run_case(sa, new, kv, 2 * G, 2, 64, 16, False, seed=G)


@pytest.mark.parametrize("new,kv", [([1] * 30 + [200], [500 + 37 * b for b in range(30)] + [900]), ([300, 1], [300, 3000]),
                                    ([1, 0, 70, 2, 0, 1], [4000, 50, 130, 2, 0, 1]), ([65, 64, 1], [65, 64, 1])])
@pytest.mark.parametrize("D,G", [(128, 4), (64, 1), (128, 16)])
@pytest.mark.parametrize("causal", [True, False])
def test_single_tokens_among_prompt_pieces(sa, new, kv, D, G, causal):
    """Sequences of few rows and of many in one call: the two forms on their own shares of the machine."""
    run_case(sa, new, kv, 2 * G, 2, D, 16, causal, seed=len(new), behind=3, holes=[(0, 1, -1)])


def test_offsets_past_32_bits(sa):
    """Pools of more than 2^32 elements: append, attend, fork and copy at their far end."""
    Hkv, ps, D, n_pages = 8, 128, 128, 33100
    assert n_pages * Hkv * ps * D > 2 ** 32
    kp = torch.empty((n_pages, Hkv, ps, D), dtype=BF, device="cuda")
    vp = torch.empty_like(kp)
    pages = [n_pages - 1, 5, n_pages - 3]
    table = i32([pages + [-1], [-1] * 4])
    refs = torch.ones(n_pages, dtype=I32, device="cuda")
    refs[[n_pages - 2, 17]] = 0
    n = 300
    lens, cu = i32([n, 0]), i32([0, n, n])
    g = torch.Generator().manual_seed(3)
    k, v, q = (torch.randn((n, H, D), generator=g).to(BF).cuda().transpose(0, 1) for H in (Hkv, Hkv, 8))
    sa.paged_append(k, v, kp, vp, table, lens, cu)
    for i, p in enumerate(pages):
        rows = min(ps, n - i * ps)
        assert torch.equal(kp[p, :, :rows], k[:, i * ps:i * ps + rows]) and torch.equal(vp[p, :, :rows], v[:, i * ps:i * ps + rows])
    dense_k, dense_v = k.contiguous()[None], v.contiguous()[None]
    got = sa.attn_paged(q, kp, vp, table, lens, cu)
    want = ref.attention(q, dense_k, dense_v, torch.zeros((1, 1), dtype=I32), torch.tensor([n]), torch.tensor([0, n]), True,
                         1 / math.sqrt(D))
    ref.check_attention(got, want)
    assert sa.paged_fork((kp, vp), table, lens, refs, [0], [1]).tolist() == [0]
    assert table[1].tolist() == [n_pages - 1, 5, 17, -1] and torch.equal(kp[17, :, :n - 256], kp[n_pages - 3, :, :n - 256])
    sa.paged_copy((kp, vp), [n_pages - 1], [n_pages - 2])
    assert torch.equal(vp[n_pages - 2], vp[n_pages - 1])


def test_after_a_timeout_the_rows_come_out_empty_until_it_is_reported(sa):
    kp, vp, table, lens, cu = make_cache([1, 3], [900, 77], 2, 128, 16, 18)
    q = torch.randn((4, 4, 128)).to(BF).cuda()
    want = sa.attn_paged(q, kp, vp, table, lens, cu)
    assert sa.lib.attn_debug_expire_wait(1000, torch.cuda.current_stream().cuda_stream) == 0
    o, lse = sa.attn_paged(q, kp, vp, table, lens, cu)
    with pytest.raises(sa.AttnError):
        sa.query_device_error()
    assert (o == 0).all() and torch.isneginf(lse).all()
    again = sa.attn_paged(q, kp, vp, table, lens, cu)
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])


def test_two_captured_calls_that_share_a_workspace_in_order(sa):
    """Two graphs with one workspace, replayed one after the other on one stream."""
    kp, vp, table, lens, cu = make_cache([1, 1], [2000, 900], 2, 128, 16, 19, garbage=False)
    qs = [torch.randn((8, 2, 128)).to(BF).cuda() for _ in range(2)]
    ws = torch.empty(sa.attn_paged_workspace_bytes(8, 2, 2, 128), dtype=torch.uint8, device="cuda")
    want = [sa.attn_paged(q, kp, vp, table, lens, cu) for q in qs]
    graphs, outs = [], []
    for q in qs:
        outs.append((torch.empty_like(q), torch.empty((8, 2), device="cuda")))
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            sa.attn_paged(q, kp, vp, table, lens, cu, out=outs[-1][0], lse=outs[-1][1], workspace=ws)
    for _ in range(5):
        for gr in graphs:
            gr.replay()
    torch.cuda.synchronize()
    for (o, lse), (wo, wl) in zip(outs, want):
        assert torch.equal(o, wo) and torch.equal(lse, wl)


# ---------------------------------------------------------------------------- rotary positions
ROPE = [(1, 1, 0, 1, 64), (2, 3, 1, 17, 64), (1, 4, 2, 131, 128), (3, 28, 4, 5, 128), (1, 2, 1, 3001, 64)]


@pytest.mark.parametrize("shape", ROPE)
@pytest.mark.parametrize("dtype", [BF, torch.float32])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_axes(sa, shape, dtype, interleaved):
    B, Hq, Hk, S, D = shape
    g = torch.Generator().manual_seed(B * S + D)
    q = torch.randn((B, Hq, S, D), generator=g).to(dtype).cuda()
    k = torch.randn((B, S, Hk, D), generator=g).to(dtype).cuda().transpose(1, 2) if Hk else None
    pos = torch.randint(-1000, 2 ** 20, (3, B, S), generator=g).to(I32).cuda()
    plan = sa.RopePlan(D, (D // 8, D // 8, D // 8 + 3))
    for fn, inverse in ((sa.rope_axes, False), (sa.rope_axes_bwd, True)):
        got = fn(q, k, pos, *plan, interleaved=interleaved)
        for x, y in zip((q, k), got):
            if x is not None:
                ref.within(y, *ref.rotate(x, pos, *plan, interleaved, inverse))
            else:
                assert y is None


def test_rope_axes_far_positions_in_place_and_shared_positions(sa):
    D = 128
    plan = sa.RopePlan(D, (64,), base=500000.0)
    x = torch.randn((2, 2, 40, D)).cuda()
    pos = torch.randint(0, 2 ** 31 - 1, (1, 1, 40)).to(I32).cuda().expand(1, 2, 40)
    want, tol = ref.rotate(x, pos, *plan, False)
    kept = x.clone()
    y, _ = sa.rope_axes(x, None, pos, *plan, out_q=x)
    assert y.data_ptr() == x.data_ptr()
    ref.within(x, want, tol)
    # turned back by the gradient: the input again, within both calls' bounds
    back, _ = sa.rope_axes_bwd(x, None, pos, *plan)
    again, tol2 = ref.rotate(x, pos, *plan, False, inverse=True)
    ref.within(back, again, tol2)
    assert (back - kept).abs().max().item() <= 4 * tol.max().item() + 4 * tol2.max().item()


def test_rope_gradient_is_the_transpose_and_matches_differences(sa):
    """<dy, R x> = <R^T dy, x>, and the difference quotient of the (linear) forward."""
    D = 64
    plan = sa.RopePlan(D, (8, 12, 12))
    g = torch.Generator().manual_seed(1)
    x, dy, v = (torch.randn((1, 2, 33, D), generator=g).cuda() for _ in range(3))
    pos = torch.randint(0, 5000, (3, 1, 33), generator=g).to(I32).cuda()
    y, _ = sa.rope_axes(x, None, pos, *plan)
    dx, _ = sa.rope_axes_bwd(dy, None, pos, *plan)
    _, t1 = ref.rotate(x, pos, *plan, False)
    _, t2 = ref.rotate(dy, pos, *plan, False, inverse=True)
    lhs, rhs = (dy.double() * y.double()).sum().item(), (dx.double() * x.double()).sum().item()
    bound = (dy.abs().double().cpu() * t1).sum().item() + (x.abs().double().cpu() * t2).sum().item()
    assert abs(lhs - rhs) <= bound
    h = 0.5  # the map is linear: any step, exact in x + h v up to one rounding of it
    x2 = x + h * v
    y2, _ = sa.rope_axes(x2, None, pos, *plan)
    _, t3 = ref.rotate(x2, pos, *plan, False)
    quotient = ((y2.double() - y.double()) * dy.double()).sum().item() / h
    slack = ((t1 + t3) * dy.abs().double().cpu()).sum().item() / h
    slack += (x2.abs().double() * dx.abs().double()).sum().item() * 2 * 2.0 ** -24 / h
    slack += (v.abs().double().cpu() * t2).sum().item()
    assert abs(quotient - (dx.double() * v.double()).sum().item()) <= slack


def test_rope_captured_backward_while_eager_results_live(sa):
    plan = sa.RopePlan(128, (16, 24, 24))
    x = torch.randn((1, 4, 100, 128)).to(BF).cuda()
    pos = torch.randint(0, 99, (3, 1, 100)).to(I32).cuda()
    eager, _ = sa.rope_axes_bwd(x, None, pos, *plan)
    out = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sa.rope_axes_bwd(x, None, pos, *plan, out_dq=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, eager)


def test_rope_of_more_than_32_bits_of_elements(sa):
    D, H, S = 128, 34, 500_000
    assert H * S * D > 2 ** 31
    plan = sa.RopePlan(D, (64,))
    x = torch.empty((1, H, S, D), dtype=BF, device="cuda").normal_()
    pos = torch.arange(S, dtype=I32, device="cuda").view(1, 1, S)
    y, _ = sa.rope_axes(x, None, pos, *plan)
    for rows in (slice(0, 3), slice(S - 40, S)):
        for h in (0, H - 1):
            ref.within(y[:, h:h + 1, rows], *ref.rotate(x[:, h:h + 1, rows], pos[:, :, rows], *plan, False))


def test_rope_rows_with_strides(sa):
    """A slice of a fused projection in, a slice of another tensor out; the rest of it untouched."""
    B, S, H, D = 2, 37, 3, 64
    fused = torch.randn((B, S, 5 * H, D)).to(BF).cuda()
    x = fused[:, :, H:2 * H].transpose(1, 2)
    out = torch.full((B, H + 2, S + 3, D), 7.0, dtype=BF, device="cuda")
    pos = torch.arange(S, dtype=I32, device="cuda").view(1, 1, S).expand(2, B, S)
    plan = sa.RopePlan(D, (16, 16), shared=False)
    y, _ = sa.rope_axes(x, None, pos, *plan, interleaved=True, out_q=out[:, 1:1 + H, 2:2 + S])
    ref.within(y, *ref.rotate(x, pos, *plan, True))
    assert (out[:, 0] == 7).all() and (out[:, H + 1] == 7).all() and (out[:, :, :2] == 7).all() and (out[:, :, S + 2] == 7).all()
    with pytest.raises(ValueError, match="expanded"):
        sa.rope_axes(x, None, pos, *plan, out_q=out[:, :1, 2:2 + S].expand(B, H, S, D))


# ---------------------------------------------------------------------------- appends
@pytest.mark.parametrize("ps,D,new,kv", [(16, 128, [1, 1, 1], [1, 16, 17]), (32, 64, [40, 0, 3], [40, 9, 65]),
                                        (128, 128, [5, 300], [130, 300]), (16, 64, [9, 6], [4, 6])])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append(sa, ps, D, new, kv, interleaved):
    """Every slot of the new tokens, and no other; tokens without a slot are dropped; rows behind the last sequence stay."""
    Hq, Hkv, behind = 6, 2, 2
    kp, vp, table, lens, cu = make_cache(new, kv, Hkv, D, ps, 21, garbage=False)
    if len(new) == 2 and new[0] == 5:
        table[1, 1] = -1
    total = sum(new) + behind
    g = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn((total, H, D), generator=g).to(BF).cuda().transpose(0, 1) for H in (Hq, Hkv, Hkv))
    pos = torch.randint(0, 10 ** 6, (3, total), generator=g).to(I32).cuda()
    plan = sa.RopePlan(D, (D // 8, D // 8, D // 4))
    want_k, want_v, tol_k = kp.double().cpu(), vp.double().cpu(), torch.full(kp.shape, 1e-30, dtype=torch.float64)
    rk, tk = ref.rotate(k[None], pos[:, None], *plan, interleaved)
    for b in range(len(new)):
        for i in range(new[b]):
            slot = kv[b] - new[b] + i
            page = int(table[b, slot // ps]) if slot >= 0 else -1
            if page < 0:
                continue
            t = sum(new[:b]) + i
            want_k[page, :, slot % ps], tol_k[page, :, slot % ps] = rk[0][:, t], tk[0][:, t]
            want_v[page, :, slot % ps] = v[:, t].double().cpu()
    out_q = torch.full((Hq, total, D), 7.0, dtype=BF, device="cuda")
    sa.paged_append(k, v, kp, vp, table, lens, cu, q=q, positions=pos, inv_freq=plan.inv_freq, axes=plan.axes,
                    interleaved=interleaved, out_q=out_q)
    ref.within(kp, want_k, tol_k)
    assert torch.equal(vp.double().cpu(), want_v)
    wq, tq = ref.rotate(q[None], pos[:, None], *plan, interleaved)
    ref.within(out_q[:, :total - behind], wq[0][:, :total - behind], tq[0][:, :total - behind])
    assert (out_q[:, total - behind:] == 7).all()
    # without positions: keys as they are
    sa.paged_append(k, v, kp, vp, table, lens, cu)
    slot = kv[0] - 1
    assert torch.equal(kp[int(table[0, slot // ps]), :, slot % ps], k[:, new[0] - 1])


# ---------------------------------------------------------------------------- page management
def tables(sa, rows, W, n_pages, ps, fill, seed, spare=3):
    """A table with `rows` filled rows of random lengths and `spare` empty ones, and its host model."""
    g = torch.Generator().manual_seed(seed)
    ids = torch.randperm(n_pages, generator=g).tolist()
    refs, table, lens, at = [0] * n_pages, [], [], 0
    for r in range(rows):
        n = min(W, max(0, int(fill * n_pages / rows) + (r % 3) - 1))
        table.append(ids[at:at + n] + [-1] * (W - n))
        at += n
        for p in table[-1][:n]:
            refs[p] = 1
        lens.append(max(0, n * ps - (r * 5) % ps))
    table += [[-1] * W for _ in range(spare)]
    lens += [0] * spare
    return i32(table), i32(lens), i32(refs), ref.Tables(table, lens, refs, ps)


def same(table, lens, refs, model):
    assert table.tolist() == model.table and lens.tolist() == model.lens and refs.tolist() == model.refs


@pytest.mark.parametrize("n_pages,rows,W,ps", [(40, 3, 9, 16), (9000, 50, 200, 32), (20011, 700, 40, 16)])
def test_reserve_and_free(sa, n_pages, rows, W, ps):
    table, lens, refs, model = tables(sa, rows, W, n_pages, ps, 0.7, rows)
    B = table.shape[0]
    for step in range(3):
        n_new = [(b * 13 + step * 5) % (3 * ps) - 2 for b in range(B)]
        status = sa.paged_reserve(table, lens, refs, i32(n_new), ps)
        assert status.tolist() == model.reserve(n_new)
        same(table, lens, refs, model)
        rows_out = list(range(step, B, 4))
        sa.paged_free(table, lens, refs, rows_out)
        model.free(rows_out)
        same(table, lens, refs, model)


def test_reserve_without_enough_pages(sa):
    """Rows are served in order while the pages last; the others stay as they are."""
    table, lens, refs, model = tables(sa, 4, 12, 20, 16, 0.6, 1)
    n_new = [30, 90, 40, 0, 200, 5, 16]
    status = sa.paged_reserve(table, lens, refs, i32(n_new), 16)
    assert status.tolist() == model.reserve(n_new) and 1 in status.tolist() and 2 in status.tolist()
    same(table, lens, refs, model)


@pytest.mark.parametrize("layered", [False, True])
def test_fork_copies_the_last_page_and_shares_the_others(sa, layered):
    ps, n_pages = 16, 300
    table, lens, refs, model = tables(sa, 5, 40, n_pages, ps, 0.5, 2, spare=8)
    lens[3] = 3 * ps  # whole pages only: nothing to copy
    model.lens[3] = 3 * ps
    shape = (3, n_pages, 2, ps, 64)
    pools = (torch.randn(shape).to(BF).cuda(), torch.randn(shape).to(BF).cuda()) if layered else \
        torch.randn(shape[1:]).cuda()
    before = [p.clone() for p in (pools if layered else (pools,))]
    src, dst = [0, 0, 3, 1, 0, 4], [5, 9, 6, 7, 12, 8]
    lens[7] = 4  # in use
    model.lens[7] = 4
    status = sa.paged_fork(pools, table, lens, refs, src, dst)
    want, copies = model.fork(src, dst)
    assert status.tolist() == want and 3 in want
    same(table, lens, refs, model)
    for p, old in zip(pools if layered else (pools,), before):
        old, layers = (old, p) if p.dim() == 5 else (old[None], p[None])
        for a, b in copies:
            old[:, b] = old[:, a]
        assert torch.equal(layers, old)


def test_fork_without_free_pages(sa):
    table, lens, refs, model = tables(sa, 2, 8, 16, 16, 0.9, 3, spare=4)
    lens[0] -= 3
    model.lens[0] -= 3
    refs[refs == 0] = 1  # all taken but one
    model.refs = [max(r, 1) for r in model.refs]
    refs[11] = model.refs[11] = 0
    pool = torch.randn((16, 1, 16, 64)).cuda()
    src, dst = [0, 0, 0], [2, 3, 4]
    assert sa.paged_fork(pool, table, lens, refs, src, dst).tolist() == model.fork(src, dst)[0] == [0, 1, 1]
    same(table, lens, refs, model)


def test_fork_and_free_more_rows_than_one_launch_takes(sa):
    ps, n_pages = 16, 3000
    table, lens, refs, model = tables(sa, 4, 10, n_pages, ps, 0.01, 4, spare=1300)
    pool = torch.randn((n_pages, 1, ps, 64)).cuda()
    src, dst = [i % 4 for i in range(1200)], list(range(4, 1204))
    assert sa.paged_fork(pool, table, lens, refs, src, dst).tolist() == model.fork(src, dst)[0]
    same(table, lens, refs, model)
    sa.paged_free(table, lens, refs, dst[1:])
    model.free(dst[1:])
    same(table, lens, refs, model)


def test_copy_pages(sa):
    n = 1500
    pools = (torch.randn((2, n, 2, 16, 64)).to(BF).cuda(), torch.randint(0, 255, (n, 1, 3, 16), dtype=torch.uint8).cuda())
    want = [p.clone() for p in pools]
    g = torch.Generator().manual_seed(0)
    ids = torch.randperm(n, generator=g).tolist()
    src, dst = ids[:600], ids[700:1300]
    src[1] = src[0]  # a source may repeat
    sa.paged_copy(pools, src, dst)
    want[0][:, dst] = want[0][:, src]
    want[1][dst] = want[1][src]
    assert all(torch.equal(a, b) for a, b in zip(pools, want))


@pytest.mark.parametrize("n_pages,rows,W,fill", [(1, 1, 4, 0.0), (40, 3, 30, 0.5), (4096, 9, 400, 0.6), (10007, 40, 300, 0.3),
                                                 (8192, 16, 512, 1.0)])
@pytest.mark.parametrize("in_place", [True, False])
def test_compact(sa, n_pages, rows, W, fill, in_place):
    table, lens, refs, model = tables(sa, rows, W, n_pages, 16, fill, n_pages)
    if rows > 3:  # shared pages count once
        table[rows] = table[0]
        model.table[rows] = list(model.table[0])
        for p in model.table[0]:
            if p >= 0:
                model.refs[p] += 1
        refs.copy_(i32(model.refs))
        table[rows + 1, 2] = 2 ** 31 - 1  # no page: stays
        model.table[rows + 1][2] = 2 ** 31 - 1
    pool = torch.randn((2, n_pages, 1, 16, 64)).to(BF).cuda()
    want = pool.clone()
    old_table, old_refs = table.clone(), refs.clone()
    out = {} if in_place else dict(out_table=torch.full_like(table, 5), out_refs=torch.full_like(refs, 5))
    n_live = sa.paged_compact(pool, table, refs, **out)
    n, moves = model.compact()
    assert n_live.item() == n
    got_t, got_r = (table, refs) if in_place else (out["out_table"], out["out_refs"])
    same(got_t, lens, got_r, model)
    if not in_place:
        assert torch.equal(table, old_table) and torch.equal(refs, old_refs)
    for a, b in moves:
        want[:, b] = want[:, a]
    assert torch.equal(pool[:, :n], want[:, :n])


# ---------------------------------------------------------------------------- together
def test_serving_steps_of_a_paged_cache(sa):
    """Prompts, forks, single tokens, a row freed and the pool compacted, then more tokens: every step's attention
    equals attention over the keys that were handed in, in order (tests keep them in a plain list per row)."""
    Hq, Hkv, D, ps, layers = 8, 2, 64, 16, 2
    plan = sa.RopePlan(D, (8, 12, 12))
    cache = sa.PagedCache(64, Hkv, D, rows=6, max_pages=12, page_size=ps, layers=layers, plan=plan)
    for p in (cache.k_pages, cache.v_pages):
        p.fill_(math.nan)
    g = torch.Generator().manual_seed(9)
    kept = {(layer, b): ([], []) for layer in range(layers) for b in range(6)}

    def step(n_new):
        assert cache.reserve(i32(n_new)).tolist() == [0] * 6
        total = sum(n_new)
        cu = [0]
        for n in n_new:
            cu.append(cu[-1] + n)
        pos = torch.stack([torch.randint(0, 999, (total,), generator=g) for _ in range(3)]).to(I32).cuda()
        for layer in range(layers):
            q, k, v = (torch.randn((total, H, D), generator=g).to(BF).cuda().transpose(0, 1) for H in (Hq, Hkv, Hkv))
            o, lse = cache.step(layer, q, k, v, i32(cu), pos)
            rq, rk = sa.rope_axes(q[None], k[None], pos[:, None], *plan)  # bitwise what the append writes
            for b, n in enumerate(n_new):
                ks, vs = kept[layer, b]
                for i in range(cu[b], cu[b + 1]):
                    ks.append(rk[0, :, i].cpu())
                    vs.append(v[:, i].cpu())
                if n == 0:
                    continue
                m = len(ks)
                dense_k, dense_v = torch.stack(ks, 1)[None], torch.stack(vs, 1)[None]  # one page of all keys
                want = ref.attention(rq[0][:, cu[b]:cu[b + 1]], dense_k, dense_v, torch.zeros((1, 1), dtype=I32),
                                     torch.tensor([m]), torch.tensor([0, n]), True, 1 / math.sqrt(D))
                ref.check_attention((o[:, cu[b]:cu[b + 1]], lse[:, cu[b]:cu[b + 1]]), want)

    def copy_rows(a, b):
        for layer in range(layers):
            kept[layer, b] = tuple(list(x) for x in kept[layer, a])

    step([37, 5, 0, 16, 0, 0])
    step([1, 1, 0, 1, 0, 0])
    assert cache.fork([0, 0, 3], [2, 4, 5]).tolist() == [0, 0, 0]
    for a, b in ((0, 2), (0, 4), (3, 5)):
        copy_rows(a, b)
    step([1, 1, 1, 1, 3, 20])
    cache.free([0, 3])
    for layer in range(layers):
        kept[layer, 0], kept[layer, 3] = ([], []), ([], [])
    before = int((cache.page_refs > 0).sum())
    assert cache.compact().item() == before and (cache.page_refs[before:] == 0).all()
    step([2, 1, 1, 0, 1, 1])
    step([1, 1, 1, 60, 1, 1])


def test_captured_serving_step(sa):
    """reserve, append and attention captured once and replayed step by step equal the same steps run directly."""
    Hq, Hkv, D = 4, 1, 128
    plan = sa.RopePlan(D, (16, 24, 24))
    caches = [sa.PagedCache(40, Hkv, D, rows=3, max_pages=9, plan=plan) for _ in range(2)]
    for c in caches:
        c.k_pages.zero_()
        c.v_pages.zero_()
    n_new, cu = i32([1, 1, 1]), i32([0, 1, 2, 3])
    q, k, v = (torch.zeros((H, 3, D), dtype=BF, device="cuda") for H in (Hq, Hkv, Hkv))
    pos = torch.zeros((3, 3), dtype=I32, device="cuda")

    def one(cache):
        cache.reserve(n_new)
        return cache.step(0, q, k, v, cu, pos)

    one(caches[0])  # warms the library up; the cache starts over
    caches[0].free([0, 1, 2])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = one(caches[0])
    for i in range(20):
        for t in (q, k, v):
            t.copy_(torch.randn(t.shape, generator=torch.Generator().manual_seed(i)).to(BF))
        pos.fill_(i)
        graph.replay()
        want = one(caches[1])
        torch.cuda.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    assert caches[0].kv_lens.tolist() == [20] * 3
    assert torch.equal(caches[0].page_table, caches[1].page_table)


def serving_chain(sa, seed, pause=lambda: None):
    """Steps of a cache whose kernels depend on one another in every way: outputs and the final state."""
    Hq, Hkv, D, ps, rows = 14, 2, 128, 16, 8
    plan = sa.RopePlan(D, (64,))
    cache = sa.PagedCache(300, Hkv, D, rows=rows, max_pages=40, page_size=ps, plan=plan)
    cache.k_pages.zero_(), cache.v_pages.zero_()
    g = torch.Generator(device="cuda").manual_seed(seed)
    outs = []
    for it in range(24):
        if it % 6 == 3:
            cache.free([4, 5, 6, 7])
            pause()
            cache.fork([0, 1, 0, 2], [4, 5, 6, 7])
            pause()
        new = [1] * rows if it % 4 else [40, 3, 70, 1] + [0] * 4
        if it % 6 < 3:
            new[4:] = [0] * 4
        n_new, cu = i32(new), torch.nn.functional.pad(i32(new).cumsum(0), (1, 0)).to(I32)
        total = sum(new)
        q, k, v = (torch.randn((H, total, D), generator=g, device="cuda").to(BF) for H in (Hq, Hkv, Hkv))
        pos = torch.randint(0, 5000, (1, total), generator=g, device="cuda", dtype=I32)
        pause()
        cache.reserve(n_new)
        pause()
        for _ in range(2):  # the second call reads what the first one read, into tensors that may be its neighbours
            outs.append(cache.step(0, q, k, v, cu, pos))
            pause()
        if it % 8 == 7:
            cache.compact()
            pause()
    return outs, (cache.page_table, cache.kv_lens, cache.page_refs)


def test_a_chain_without_waits_equals_one_with_waits(sa):
    """Every kernel may start before the one ahead of it has ended; none may read or write too early."""
    want, state = serving_chain(sa, 3, torch.cuda.synchronize)
    for _ in range(3):
        got, after = serving_chain(sa, 3)
        for (o, lse), (wo, wl) in zip(got, want):
            assert torch.equal(o, wo) and torch.equal(lse, wl)
        for a, b in zip(after, state):
            assert torch.equal(a, b)


def test_chains_on_two_streams_at_once(sa):
    want = [serving_chain(sa, s, torch.cuda.synchronize)[0] for s in (5, 6)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for s, stream in zip((5, 6), streams):
        with torch.cuda.stream(stream):
            got.append(serving_chain(sa, s)[0])
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        for (o, lse), (wo, wl) in zip(a, b):
            assert torch.equal(o, wo) and torch.equal(lse, wl)

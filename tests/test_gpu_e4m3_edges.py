"""The 8-bit cache where its kernels hand work from one warpgroup to the other, and where weights and values lie far
apart (bounds: e4m3_ref.py)."""
import math

import pytest
import torch

from tests import drafts_ref, e4m3_ref
from tests.test_gpu_drafts import Cache, queries, sa  # noqa: F401
from tests.test_gpu_paged import i32

pytestmark = pytest.mark.gpu
BF, I32, U8 = torch.bfloat16, torch.int32, torch.uint8
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


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


class OneContext:
    """A context of n keys that B sequences share, page by page, so that an item of one CTA goes through all of it: keys and
    values in fp64 [Hkv, n, D], as codes in the pools, and B * q_len queries with a common direction, which no key has a
    part in until one is given it."""

    def __init__(self, n, B, q_len, G, D, Hkv=2, seed=0):
        g = torch.Generator().manual_seed(seed)
        self.n, self.B, self.q_len, self.G, self.Hkv, self.D = n, B, q_len, G, Hkv, D
        self.u = torch.ones(D, dtype=torch.float64) / math.sqrt(D)
        k, self.v = (torch.randn((Hkv, n, D), generator=g).double() for _ in range(2))
        self.k = k - (k @ self.u)[..., None] * self.u
        q = torch.randn((B * q_len, Hkv * G, D), generator=g).double()
        q = q - (q @ self.u)[..., None] * self.u + math.sqrt(D) * self.u
        self.q = q.to(BF).cuda().transpose(0, 1)
        self.order = torch.randperm(n // 16, generator=g)

    def raise_key(self, i, nats):
        """Key i's score of every row is about `nats` (others: normal, about 1)."""
        self.k[:, i] = self.u * nats

    def fill(self):
        pools, scales, self.values, self.exps, self.codes = [], [], [], [], []
        for x in (self.k, self.v):
            codes, sc = drafts_ref.quantise(x)
            self.values.append(drafts_ref.values(codes, sc).cuda())
            self.exps.append(e4m3_ref.exponents(sc).cuda())
            self.codes.append(codes.float().cuda())
            p = torch.empty((self.n // 16, self.Hkv, 16, self.D), dtype=U8)
            p[self.order] = codes.view(U8).reshape(self.Hkv, -1, 16, self.D).transpose(0, 1)
            s = torch.empty((self.n // 16, self.Hkv, 16), dtype=U8)
            s[self.order] = sc.view(U8).reshape(self.Hkv, -1, 16).transpose(0, 1)
            pools.append(p.cuda().view(E4M3))
            scales.append(s.cuda().view(E8M0))
        self.pools, self.kw = pools, {"k_scales": scales[0], "v_scales": scales[1]}
        self.table = self.order.to(I32).repeat(self.B, 1).cuda()
        self.lens, self.cu = i32([self.n] * self.B), i32([b * self.q_len for b in range(self.B + 1)])

    def check(self, sa, picked=(0, 17), tree=None, seen_new=None, least=2.0 ** -7):  # noqa: F811
        """Every element within its bound; and a row's error, as a whole, within `least` of the row: a weight's rounding error of
        at most 2^-9, of either sign, adds up over keys as the row itself does, to about 2^-10 of it, the row's own rounding
        is as much again, and what a form loses of a score far above 1 less; 2^-7 is four times all of it. On top of it the wide
        form is granted what its first tile's floor can take: each weight at most itself, and 2^-38 of the largest (with 30
        nats, 2^43, between them, all that the sink's 127 neighbours bring); and what values beside far larger ones can lose."""
        o, lse = sa.attn_paged(self.q, *self.pools, self.table, self.lens, self.cu, tree=tree, **self.kw)
        again = sa.attn_paged(self.q, *self.pools, self.table, self.lens, self.cu, tree=tree, **self.kw)
        assert torch.equal(o, again[0]) and torch.equal(lse, again[1])
        draft = torch.arange(self.n, device="cuda") - (self.n - self.q_len)
        own = torch.ones((self.q_len, self.q_len), dtype=torch.bool).tril().cuda() if seen_new is None else seen_new
        seen = (draft < 0)[None, :] | own[:, draft.clamp(min=0)]
        seen = seen.repeat_interleave(self.G, 0)
        wide = self.q_len * self.G > 64
        for b in picked:
            for h in range(self.Hkv):
                heads, rows = slice(h * self.G, (h + 1) * self.G), slice(b * self.q_len, (b + 1) * self.q_len)
                flat = lambda x: x[heads, rows].transpose(0, 1).reshape(self.q_len * self.G, *x.shape[2:]).double()  # noqa: E731
                r = e4m3_ref.attention(flat(self.q), self.values[0][h], self.values[1][h], self.exps[0][h], self.exps[1][h],
                                       self.codes[1][h], seen, 1 / math.sqrt(self.D), wide)
                got, got_lse = flat(o), flat(lse)
                assert ((got - r[0]).abs() <= r[1]).all(), float(((got - r[0]).abs() / r[1]).max())
                assert ((got_lse - r[2]).abs() <= r[3]).all()
                off = (got - r[0]).norm(dim=-1) / r[0].norm(dim=-1).clamp(min=1e-300)
                assert (off <= least + r[4]).all(), float((off - r[4]).max())


# rows of a KV head in each form: 1 and 16 (tiles in turn), 32, 64, and 160 (wide)
FORMS = [(1, 1), (4, 4), (2, 16), (8, 8), (40, 4)]


@pytest.mark.parametrize("q_len,G", FORMS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,nats,size", [(8192, 12.0, 0.0), (8192, 30.0, 2.0 ** -60), (16384, 14.0, 2.0 ** -10), (65536, 16.0, 0.0), (4096, 10.0, 0.01),
                                         (16384, 20.0, 0.0)])
def test_a_first_key_that_takes_most_of_the_weight(sa, q_len, G, D, n, nats, size):  # noqa: F811
    """A sink: its value is small or zero, and what the other keys' small weights bring is the answer."""
    c = OneContext(n, 200, q_len, G, D, seed=n + D)
    c.raise_key(0, nats)
    c.v[:, 0] *= size
    c.fill()
    c.check(sa)


@pytest.mark.parametrize("q_len,G", FORMS)
@pytest.mark.parametrize("bits", [8, 12, 20])
@pytest.mark.parametrize("sink", [None, 13.0])
def test_one_value_far_larger_than_the_others_and_of_no_weight(sa, q_len, G, bits, sink):  # noqa: F811
    """Its scale must not take bits from the other keys, in its own tile and behind it, with a sink and without."""
    c = OneContext(16384, 200, q_len, G, 128, seed=bits)
    for i in (37, 5000):
        c.raise_key(i, -120.0)
        c.v[:, i] *= 2.0 ** bits
    if sink is not None:
        c.raise_key(0, sink)
        c.v[:, 0] = 0
    c.fill()
    c.check(sa)


@pytest.mark.parametrize("q_len,G", FORMS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("of_keys", [False, True])
def test_scales_that_lie_further_apart_than_fp16_in_one_tile(sa, q_len, G, D, of_keys):  # noqa: F811
    """Keys of no weight whose value, or which themselves, are about 2^26 to 2^29 above all others of their tile: these keep
    what fp16 can hold of them."""
    c = OneContext(2048, 200, q_len, G, D, seed=3)
    for n, i in enumerate((37, 300, 700, 1500, 1999)):
        c.raise_key(i, -120.0)
        if of_keys:
            c.k[:, i] *= 2.0 ** 23  # elements of 120 / sqrt(D) against others of about 1
        else:
            c.v[:, i] *= 2.0 ** (26 + n % 4)
    c.fill()
    c.check(sa)


@pytest.mark.parametrize("q_len,G", FORMS)
@pytest.mark.parametrize("bits", [16, 21, 23, 24, 25, 26, 27, 28, 30, 40])
@pytest.mark.parametrize("spread", [0, 46, 60])
def test_scores_whose_steps_are_larger_than_any_headroom(sa, q_len, G, bits, spread):  # noqa: F811
    """Scores of 2^18 and far more, in every sequence other ones, so that references are rounded to steps of up to 2^20; values
    of one size and of two that lie far apart. Everything within its bound, and so finite."""
    c = OneContext(1024, 160, q_len, G, 128, seed=bits)
    sizes = 2.0 ** (bits - 3 * torch.rand(c.q.shape[1], generator=torch.Generator().manual_seed(bits)))
    c.q = (c.q * sizes.cuda()[None, :, None]).to(BF)
    c.v[:, torch.arange(c.n) % 3 > 0] *= 2.0 ** -spread
    c.fill()
    c.check(sa, picked=range(0, 160, 9), least=math.inf)
    o, lse = sa.attn_paged(c.q, *c.pools, c.table, c.lens, c.cu, **c.kw)
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("q_len,G", FORMS)
def test_weights_that_fall_and_rise_over_the_tiles(sa, q_len, G):  # noqa: F811
    """Tiles of large and of small weights in turn, the large ones with values of next to nothing; sizes of values that
    come and go."""
    c = OneContext(8192, 200, q_len, G, 128, seed=5)
    for t in range(0, 64, 3):
        c.raise_key(128 * t + 11, 9.0 + t / 8)
        c.v[:, 128 * t + 11] *= 2.0 ** -30
    for t in range(64):
        c.v[:, 128 * t:128 * t + 128] *= 2.0 ** (-14 if t % 7 == 3 else 0)
    c.fill()
    c.check(sa)


@pytest.mark.parametrize("q_len,G,bits", [(4, 4, 12), (4, 4, 60), (8, 8, 12), (8, 8, 60), (40, 4, 12), (40, 4, 20)])
def test_drafts_of_another_branch_take_no_bits(sa, q_len, G, bits):  # noqa: F811
    """The second half of the drafts has values far larger than all others; the first half does not see them."""
    c = OneContext(2048, 200, q_len, G, 128, seed=bits)
    half, first = q_len // 2, c.n - q_len
    c.v[:, first + half:] *= 2.0 ** bits
    c.fill()
    own = torch.zeros((q_len, q_len), dtype=torch.bool)
    own[:half, :half] = torch.ones((half, half), dtype=torch.bool).tril()
    own[half:, half:] = torch.ones((q_len - half, q_len - half), dtype=torch.bool).tril()
    bits_of = [[sum(1 << i for i in range(q_len) if own[t, i])] for t in range(q_len)] * c.B
    c.check(sa, tree=torch.tensor(bits_of, dtype=torch.int64).cuda(), seen_new=own.cuda())


def test_infinities_and_the_largest_numbers_are_read_as_infinities(sa):  # noqa: F811
    """448 2^120 is past fp32 and bf16, and so is 256 2^120, the nearest code to bf16's largest numbers. Other rows and the
    row's NaN do not notice."""
    D, n = 128, 5
    x = torch.randn((1, n, D), generator=torch.Generator().manual_seed(3)).to(BF)
    x[0, 0, 3], x[0, 0, 4], x[0, 0, 5] = math.inf, -math.inf, math.nan
    x[0, 1, 7], x[0, 1, 8], x[0, 1, 9] = torch.finfo(BF).max, 247 * 2.0 ** 120, -240 * 2.0 ** 120
    x[0, 3, 0] = -math.inf
    pools = [torch.zeros((1, 1, 16, D), dtype=U8, device="cuda").view(E4M3) for _ in range(2)]
    scales = [torch.zeros((1, 1, 16), dtype=U8, device="cuda").view(E8M0) for _ in range(2)]
    at = i32([[0]]), i32([n]), i32([0, n])
    sa.paged_append(x.cuda(), x.cuda(), *pools, *at, k_scales=scales[0], v_scales=scales[1])
    for out in sa.paged_read(*pools, *at, n, k_scales=scales[0], v_scales=scales[1]):
        out = out[0].cpu()
        assert out[0, 3] == math.inf and out[0, 4] == -math.inf and out[0, 5].isnan() and (out[0, 6:] == 0).all()
        assert out[1, 7] == math.inf and out[1, 8] == 240 * 2.0 ** 120 and out[1, 9] == -240 * 2.0 ** 120
        assert out[3, 0] == -math.inf and (out[3, 1:] == 0).all()
        for i in (2, 4):
            assert torch.equal(out[i].double(), drafts_ref.values(*drafts_ref.quantise(x[0, i].float())))

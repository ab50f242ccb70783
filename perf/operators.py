"""Cases of the paged-cache and rotary-position operators: attention over a paged cache, rotary
positions with several axes and their gradient, appending new tokens to the cache, and the page
management of the cache (forking, freeing and reserving, compacting).

``listed()`` and ``draw(rng)`` give cases, ``prepare`` makes a case's inputs on the GPU, ``run``
takes one pass through the operator (through the package where ``own`` is true, else in plain
torch operations), ``work`` counts what the pass cannot do without, and ``exact`` computes the same
outputs in 64 bits."""
import math

import torch

own = False

I32, I64, F32, F64, BF16 = torch.int32, torch.int64, torch.float32, torch.float64, torch.bfloat16


# ---------------------------------------------------------------------------- cases
def attn(name, B, Hq, Hkv, D, ps, new, ctx, causal=True, evicted=0.0, token_major=True):
    """B sequences of new[0]..new[1] new tokens behind ctx[0]..ctx[1] cached ones."""
    return {"name": name, "op": "attn", "B": B, "Hq": Hq, "Hkv": Hkv, "D": D, "ps": ps, "new_lo": new[0],
            "new_hi": new[1], "ctx_lo": ctx[0], "ctx_hi": ctx[1], "causal": causal, "evicted": evicted,
            "token_major": token_major}


def append(name, B, Hq, Hkv, D, ps, new, ctx, interleaved=False):
    return {"name": name, "op": "append", "B": B, "Hq": Hq, "Hkv": Hkv, "D": D, "ps": ps, "new_lo": new[0],
            "new_hi": new[1], "ctx_lo": ctx[0], "ctx_hi": ctx[1], "interleaved": interleaved}


def rope(name, B, Hq, Hkv, S, D, dtype, interleaved=False):
    return {"name": name, "op": "rope", "B": B, "Hq": Hq, "Hkv": Hkv, "S": S, "D": D, "dtype": dtype,
            "interleaved": interleaved}


def pages(name, op, pools, n_pages, Hkv, ps, D, rows, fill, count):
    """op "fork": count forks of the rows of a table; "compact": a pool of which `fill` is live."""
    return {"name": name, "op": op, "pools": pools, "n_pages": n_pages, "Hkv": Hkv, "ps": ps, "D": D, "rows": rows,
            "fill": fill, "count": count}


def listed():
    return [
        # one conversation's next token, short cache: the latency of a call
        attn("decode_one", 1, 28, 4, 128, 16, (1, 1), (517, 517)),
        # a serving batch's next tokens, ragged contexts: the cache is read once
        attn("decode_batch", 64, 32, 8, 128, 64, (1, 1), (300, 16000)),
        # next token of a few long sequences whose middle pages were evicted, and a draft of up to 6 to check
        attn("decode_evicted", 3, 28, 4, 128, 32, (2, 6), (40000, 131000), evicted=0.25, token_major=False),
        # a mixed batch: some sequences decode, others bring a piece of their prompt
        attn("chunk_mixed", 6, 28, 4, 128, 16, (1, 700), (100, 12000)),
        # one piece of a long prompt behind a long cache: compute bound
        attn("chunk_long", 1, 32, 8, 128, 128, (1024, 1024), (65536, 65536)),
        # an encoder's queries over all cached keys of small heads, no mask
        attn("cross_d64", 4, 8, 8, 64, 16, (130, 700), (1000, 3100), causal=False, token_major=False),
        # one token of each sequence of a serving batch into the cache: latency
        append("append_decode", 64, 32, 8, 128, 64, (1, 1), (300, 4000)),
        # a prompt piece of several sequences into the cache
        append("append_chunk", 5, 28, 4, 128, 16, (700, 3300), (0, 2000), interleaved=True),
        # rotary positions of a small image model in fp32
        rope("rope_small", 2, 8, 2, 77, 64, "float32", interleaved=True),
        # rotary positions of a long training sequence and their gradient
        rope("rope_train", 1, 28, 4, 32768, 128, "bfloat16"),
        # several answers to each prompt: children freed, forked again and given room for their next tokens
        pages("fork_cycle", "fork", 16, 4096, 4, 16, 128, 40, 0.6, 100),
        # a fragmented pool made dense
        pages("compact_pool", "compact", 8, 4096, 8, 32, 128, 64, 0.6, 0),
    ]


def spread(rng, lo, hi):
    """A size between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    case = drawn(rng)
    del case["name"]
    return case


def drawn(rng):
    op = rng.choice(["attn", "attn", "attn", "append", "rope", "fork", "compact"])
    D = rng.choice([64, 128, 128])
    ps = rng.choice([16, 32, 64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 7, 8]) if Hkv < 8 else Hkv * rng.choice([1, 2, 4])
    if op == "attn":
        B = spread(rng, 1, 48)
        new_hi = spread(rng, 1, 900) if rng.random() < 0.6 else 1
        ctx_hi = spread(rng, 64, max(256, 48000 // max(1, B * new_hi // 64 + B // 8)))
        return attn("drawn", B, Hq, Hkv, D, ps, (max(1, int(new_hi * rng.random())), new_hi),
                    (int(ctx_hi * rng.random()), ctx_hi), rng.random() < 0.8, rng.choice([0.0, 0.0, 0.3]),
                    rng.random() < 0.5)
    if op == "append":
        B = spread(rng, 1, 64)
        new_hi = spread(rng, 1, 9000 // B)
        ctx_hi = spread(rng, 1, 3000)
        return append("drawn", B, Hq, Hkv, D, ps, (max(1, int(new_hi * rng.random())), new_hi),
                      (int(ctx_hi * rng.random()), ctx_hi), rng.random() < 0.5)
    if op == "rope":
        B = rng.choice([1, 2, 3])
        return rope("drawn", B, Hq, Hkv, spread(rng, 1, 30000 // B), D, rng.choice(["bfloat16", "bfloat16", "float32"]),
                    rng.random() < 0.5)
    pools = rng.choice([1, 2, 4, 8])
    n_pages = spread(rng, 300, 4000)
    fill = rng.uniform(0.2, 0.7)
    if op == "fork":
        return pages("drawn", op, pools, n_pages, rng.choice([1, 2, 4]), rng.choice([16, 32]), D, spread(rng, 2, 60), fill,
                     spread(rng, 1, n_pages // 8))
    return pages("drawn", op, pools, n_pages, rng.choice([1, 2, 4, 8]), rng.choice([16, 32]), D, spread(rng, 1, 60),
                 fill, 0)


def lengths(c):
    """(new tokens, cached tokens before them) of each sequence, host lists."""
    new, ctx = [], []
    for b in range(c["B"]):
        f, g = ((b + 1) * 0.6180339887) % 1.0, ((b + 1) * 0.7548776662) % 1.0
        new.append(c["new_lo"] + int(round(f * (c["new_hi"] - c["new_lo"]))))
        ctx.append(c["ctx_hi"] - int(round((1.0 - g) * (c["ctx_hi"] - c["ctx_lo"]))) if b else c["ctx_hi"])
    return new, ctx


def axis_of_pairs(D):
    """Axis (time, height, width) of each of the D / 2 rotary pairs: a quarter, three eighths, three eighths."""
    half = D // 2
    a, b = half // 4, half // 4 + (half * 3) // 8
    return [0 if i < a else 1 if i < b else 2 for i in range(half)]


# ---------------------------------------------------------------------------- inputs
def normal(g, shape, dtype=BF16):
    return torch.randn(shape, generator=g, device="cuda", dtype=F32 if dtype == F32 else BF16)


def positions(c, g, n):
    """[3, n] positions as of text with images between: time runs on, height and width count in 24-wide grids
    of some stretches."""
    at = torch.arange(n, device="cuda")
    start = torch.randint(0, 1_000_000, (1,), generator=g, device="cuda")
    image = (at // 96) % 3 == 1
    t = torch.where(image, at // 96 * 96, at) + start
    h = torch.where(image, t + (at % 96) // 24, t)
    w = torch.where(image, t + at % 24, t)
    return torch.stack([t, h, w]).to(I32)


def rotary(c, s):
    D = c["D"]
    s["inv_freq"] = torch.tensor([10000.0 ** (-2.0 * i / D) for i in range(D // 2)], dtype=F64)
    s["axes"] = torch.tensor(axis_of_pairs(D), dtype=I32)
    s["inv_freq_dev"], s["axes_dev"] = s["inv_freq"].cuda(), s["axes"].cuda().long()


def cache(c, g, s):
    """Pools, page table, lengths and packed-sequence offsets of a batch; the new tokens have their pages already."""
    new, ctx = lengths(c)
    ps, B = c["ps"], c["B"]
    kv = [n + x for n, x in zip(new, ctx)]
    n_pages_of = [-(-x // ps) for x in kv]
    total_pages = sum(n_pages_of) + 7
    width = max(n_pages_of) + 3
    ids = torch.randperm(total_pages, generator=g, device="cuda").to(I32).cpu()
    table = torch.full((B, width), -1, dtype=I32)
    at = 0
    for b, n in enumerate(n_pages_of):
        table[b, :n] = ids[at:at + n]
        at += n
    if c.get("evicted"):  # pages of the middle, given up: no page any more
        for b, n in enumerate(n_pages_of):
            lo = n // 4
            table[b, lo:lo + int(c["evicted"] * ctx[b] / ps)] = -1
    shape = (total_pages, c["Hkv"], ps, c["D"])
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s.update(k_pages=normal(g, shape), v_pages=normal(g, shape), table=table.cuda(),
             kv_lens=torch.tensor(kv, dtype=I32, device="cuda"), cu=torch.tensor(cu, dtype=I32, device="cuda"),
             total=cu[-1], max_new=max(new), max_kv=max(kv))


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 13)
    s = {"c": c}
    if c["op"] == "attn":
        cache(c, g, s)
        q = normal(g, (s["total"], c["Hq"], c["D"]) if c["token_major"] else (c["Hq"], s["total"], c["D"]))
        s["q"] = q.transpose(0, 1) if c["token_major"] else q
    elif c["op"] == "append":
        cache(c, g, s)
        rotary(c, s)
        s["q"] = normal(g, (s["total"], c["Hq"], c["D"])).transpose(0, 1)
        s["k"] = normal(g, (s["total"], c["Hkv"], c["D"])).transpose(0, 1)
        s["v"] = normal(g, (s["total"], c["Hkv"], c["D"])).transpose(0, 1)
        s["pos"] = positions(c, g, s["total"])
    elif c["op"] == "rope":
        dt = F32 if c["dtype"] == "float32" else BF16
        rotary(c, s)
        for n, H in (("q", c["Hq"]), ("k", c["Hkv"]), ("dq", c["Hq"]), ("dk", c["Hkv"])):
            s[n] = normal(g, (c["B"], H, c["S"], c["D"]), dt)
        s["pos"] = torch.stack([positions(c, g, c["S"]) for _ in range(c["B"])], 1).contiguous()
    else:
        page_state(c, g, s)
    return s


def page_state(c, g, s):
    n, ps, rows = c["n_pages"], c["ps"], c["rows"]
    s["pool"] = normal(g, (c["pools"], n, c["Hkv"], ps, c["D"]))
    live = max(rows, int(c["fill"] * n))
    ids = torch.randperm(n, generator=g, device="cuda").to(I32).cpu()
    # the live pages, dealt over the rows of the table; every row's last page is partly filled
    each = [live // rows + (1 if r < live % rows else 0) for r in range(rows)]
    kids = c["count"] if c["op"] == "fork" else 0
    width = max(each) + 4
    table = torch.full((rows + kids, width), -1, dtype=I32)
    lens = torch.zeros(rows + kids, dtype=I32)
    at = 0
    for r, k in enumerate(each):
        table[r, :k] = ids[at:at + k]
        at += k
        lens[r] = k * ps - 1 - (r * 5) % (ps - 1)
    refs = torch.zeros(n, dtype=I32)
    refs[ids[:at].long()] = 1
    s.update(table=table.cuda(), lens=lens.cuda(), refs=refs.cuda())
    if c["op"] == "fork":
        s["src"] = torch.tensor([r % rows for r in range(kids)], dtype=I32)
        s["dst"] = torch.tensor([rows + r for r in range(kids)], dtype=I32)
        # the children's next tokens: one, or a draft of up to six
        s["n_new"] = torch.tensor([0] * rows + [1 + r % 6 for r in range(kids)], dtype=I32).cuda()
        s["status"] = torch.zeros(kids, dtype=I32, device="cuda")
        s["status_new"] = torch.zeros(rows + kids, dtype=I32, device="cuda")
    else:
        s.update(out_table=torch.zeros_like(s["table"]), out_refs=torch.zeros_like(s["refs"]))


# ---------------------------------------------------------------------------- one pass
def run(state):
    return (run_own if own else run_plain)(state)


def run_own(s):
    import sequence_attn_fwd_gb300 as sa

    c, op = s["c"], s["c"]["op"]
    if op == "attn":
        return sa.attn_paged(s["q"], s["k_pages"], s["v_pages"], s["table"], s["kv_lens"], s["cu"], causal=c["causal"])
    if op == "append":
        q = sa.paged_append(s["k"], s["v"], s["k_pages"], s["v_pages"], s["table"], s["kv_lens"], s["cu"], q=s["q"],
                            positions=s["pos"], inv_freq=s["inv_freq"], axes=s["axes"], interleaved=c["interleaved"])
        return q, s["k_pages"], s["v_pages"]
    if op == "rope":
        y = sa.rope_axes(s["q"], s["k"], s["pos"], s["inv_freq"], s["axes"], interleaved=c["interleaved"])
        dx = sa.rope_axes_bwd(s["dq"], s["dk"], s["pos"], s["inv_freq"], s["axes"], interleaved=c["interleaved"])
        return y, dx
    if op == "fork":
        sa.paged_free(s["table"], s["lens"], s["refs"], s["dst"])
        sa.paged_fork(s["pool"], s["table"], s["lens"], s["refs"], s["src"], s["dst"], status=s["status"])
        sa.paged_reserve(s["table"], s["lens"], s["refs"], s["n_new"], c["ps"], status=s["status_new"])
        return s["pool"], s["table"], s["lens"], s["refs"], s["status"], s["status_new"]
    n_live = sa.paged_compact(s["pool"], s["table"], s["refs"], out_table=s["out_table"], out_refs=s["out_refs"])
    return s["pool"], s["out_table"], s["out_refs"], n_live


def run_plain(s):
    return {"attn": plain_attn, "append": plain_append, "rope": plain_rope, "fork": plain_fork,
            "compact": plain_compact}[s["c"]["op"]](s)


def plain_attn(s):
    """Sequences padded to the longest; scores, masks and sums in fp32."""
    c = s["c"]
    Hkv, G, D, ps, B = c["Hkv"], c["Hq"] // c["Hkv"], c["D"], c["ps"], c["B"]
    T, S, total = s["max_new"], s["max_kv"], s["total"]
    cu, kv = s["cu"].long(), s["kv_lens"].long()
    new = cu[1:] - cu[:-1]
    t, j = torch.arange(T, device="cuda"), torch.arange(S, device="cuda")
    token = torch.where(t < new[:, None], cu[:-1, None] + t, total)                 # [B, T]; total: none
    page = s["table"].long()[:, j // ps]                                          # [B, S]
    there = (page >= 0) & (page < s["k_pages"].shape[0]) & (j < kv[:, None])
    page = torch.where(there, page, 0)
    k = s["k_pages"][page, :, j % ps].float().permute(0, 2, 3, 1)                 # [B, Hkv, D, S]
    v = torch.where(there[:, :, None, None], s["v_pages"][page, :, j % ps].float(), 0.0).permute(0, 2, 1, 3)
    q = s["q"][:, token.clamp(max=total - 1)].float()                             # [Hq, B, T, D]
    q = q.reshape(Hkv, G, B, T, D).permute(2, 0, 1, 3, 4).reshape(B, Hkv, G * T, D)
    seen = there[:, None, :].expand(B, T, S)
    if c["causal"]:
        seen = seen & (j <= (kv - new)[:, None, None] + t[:, None])
    x = (torch.matmul(q, k) * (1.0 / math.sqrt(D))).reshape(B, Hkv, G, T, S)
    x = x.masked_fill_(~seen[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    x = x.sub_(m).exp_()
    sums = x.sum(-1, keepdim=True)
    o = torch.matmul(x.reshape(B, Hkv, G * T, S), v).reshape(B, Hkv, G, T, D)
    o = torch.where(sums > 0, o / sums, 0.0)
    lse = (m + sums.log())[..., 0]
    out = torch.zeros((c["Hq"], total + 1, D), dtype=BF16, device="cuda")
    out_lse = torch.zeros((c["Hq"], total + 1), dtype=F32, device="cuda")
    out[:, token] = o.permute(1, 2, 0, 3, 4).reshape(c["Hq"], B, T, D).to(BF16)
    out_lse[:, token] = lse.permute(1, 2, 0, 3).reshape(c["Hq"], B, T)
    return out[:, :total], out_lse[:, :total]


def rotate(x, pos, s, sign):
    """x [..., n, D] rotated by the angles of pos [3, ..., n] (heads are the dimension before n)."""
    c = s["c"]
    angle = pos.double().movedim(0, -1)[..., s["axes_dev"]] * s["inv_freq_dev"]  # 64 bits: far positions
    cos, sin = angle.cos().float(), sign * angle.sin().float()
    x32 = x.float()
    if c["interleaved"]:
        a, b = x32[..., 0::2], x32[..., 1::2]
        return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2).to(x.dtype)
    a, b = x32.chunk(2, -1)
    return torch.cat([a * cos - b * sin, a * sin + b * cos], -1).to(x.dtype)


def plain_rope(s):
    pos = s["pos"][:, :, None]  # [3, B, 1, S]
    return ((rotate(s["q"], pos, s, 1.0), rotate(s["k"], pos, s, 1.0)),
            (rotate(s["dq"], pos, s, -1.0), rotate(s["dk"], pos, s, -1.0)))


def plain_append(s):
    c = s["c"]
    cu, kv = s["cu"].long(), s["kv_lens"].long()
    token = torch.arange(s["total"], device="cuda")
    b = torch.searchsorted(cu, token, right=True) - 1
    slot = kv[b] - (cu[b + 1] - token)
    page = s["table"].long()[b, slot // c["ps"]]
    s["k_pages"][page, :, slot % c["ps"]] = rotate(s["k"], s["pos"], s, 1.0).transpose(0, 1)
    s["v_pages"][page, :, slot % c["ps"]] = s["v"].transpose(0, 1)
    return rotate(s["q"], s["pos"], s, 1.0), s["k_pages"], s["v_pages"]


def plain_free(s, rows):
    n = s["refs"].numel()
    e = s["table"][rows].long()
    held = (e >= 0) & (e < n)
    refs = torch.cat([s["refs"], s["refs"].new_zeros(1)])
    refs.index_add_(0, torch.where(held, e, n).reshape(-1), -held.reshape(-1).to(I32))
    s["refs"].copy_(refs[:n])
    s["table"][rows] = -1
    s["lens"][rows] = 0


def free_pages(refs):
    """Page ids, the free ones first, each part in ascending order."""
    return torch.argsort((refs != 0).to(torch.uint8), stable=True)


def plain_fork(s):
    c, n = s["c"], s["c"]["n_pages"]
    ps = c["ps"]
    src, dst = s["src"].cuda().long(), s["dst"].cuda().long()
    plain_free(s, dst)
    table, lens, refs = s["table"], s["lens"], s["refs"]
    col = torch.arange(table.shape[1], device="cuda")
    # forks: whole pages shared, the partly filled last one copied
    length = lens[src].long()
    whole, part = length // ps, length % ps > 0
    mine = free_pages(refs)[(part.cumsum(0) - 1).clamp(min=0)]
    row = table[src].long()
    tail = row.gather(1, whole.clamp(max=table.shape[1] - 1)[:, None])[:, 0]
    shared = col < whole[:, None]
    table[dst] = torch.where(shared, row, torch.where((col == whole[:, None]) & part[:, None], mine[:, None], -1)).to(I32)
    lens[dst] = length.to(I32)
    more = torch.zeros(n + 1, dtype=I32, device="cuda")
    more.index_add_(0, torch.where(shared, row, n).reshape(-1), shared.reshape(-1).to(I32))
    more.index_add_(0, torch.where(part, mine, n), part.to(I32))
    refs += more[:n]
    to, frm = torch.where(part, mine, row[:, 0]), torch.where(part, tail, row[:, 0])
    s["pool"][:, to] = s["pool"][:, frm]
    # room for the new tokens of every row
    have, want = (lens + ps - 1) // ps, (lens + s["n_new"] + ps - 1) // ps
    need = want - have
    fresh = (col >= have[:, None]) & (col < want[:, None])
    rank = (need.cumsum(0) - need)[:, None] + col - have[:, None]
    page = free_pages(refs)[rank.clamp(0, n - 1)]
    table.copy_(torch.where(fresh, page, table.long()).to(I32))
    more = torch.zeros(n + 1, dtype=I32, device="cuda")
    more.index_add_(0, torch.where(fresh, page, n).reshape(-1), fresh.reshape(-1).to(I32))
    refs += more[:n]
    lens += s["n_new"]
    return s["pool"], table, lens, refs, torch.zeros_like(s["status"]), torch.zeros_like(s["status_new"])


def plain_compact(s):
    n = s["c"]["n_pages"]
    refs, at = s["refs"], torch.arange(n, device="cuda")
    live = refs > 0
    n_live = live.sum()
    above, hole = live & (at >= n_live), ~live & (at < n_live)
    src, dst = above.nonzero()[:, 0], hole.nonzero()[:, 0]
    to = at.clone()
    to[src] = dst
    e = s["table"].long()
    held = (e >= 0) & (e < n)
    table = torch.where(held, to[e.clamp(0, n - 1)], e).to(I32)
    out_refs = torch.zeros_like(refs).index_add_(0, to, refs)
    s["pool"][:, dst] = s["pool"][:, src]
    return s["pool"], table, out_refs, n_live.to(I32).reshape(1)


# ---------------------------------------------------------------------------- what a pass needs
def kept(c, b, n_keys, ctx):
    """Keys of sequence b that have a page."""
    return n_keys - int(c.get("evicted", 0.0) * ctx / c["ps"]) * c["ps"]


def work(case):
    c = case
    if c["op"] in ("attn", "append"):
        new, ctx = lengths(c)
        total = sum(new)
    if c["op"] == "attn":
        D, keys, pairs = c["D"], 0, 0.0
        for b, (n, x) in enumerate(zip(new, ctx)):
            k = kept(c, b, n + x, x)
            keys += k
            pairs += n * k - (n * (n - 1) / 2 if c["causal"] else 0)
        return {"bytes": 4 * D * c["Hkv"] * keys + total * c["Hq"] * (4 * D + 4), "flops": 4.0 * D * c["Hq"] * pairs}
    if c["op"] == "append":
        heads = c["Hq"] + 2 * c["Hkv"]
        return {"bytes": total * (heads * c["D"] * 4 + 12), "flops": 6.0 * total * (c["Hq"] + c["Hkv"]) * c["D"] / 2}
    if c["op"] == "rope":
        n = c["B"] * c["S"] * (c["Hq"] + c["Hkv"]) * c["D"]
        return {"bytes": 2 * n * 2 * (4 if c["dtype"] == "float32" else 2) + 12 * c["B"] * c["S"], "flops": 2 * 6.0 * n / 2}
    page = c["Hkv"] * c["ps"] * c["D"] * 2
    live = max(c["rows"], int(c["fill"] * c["n_pages"]))
    if c["op"] == "fork":
        entries = c["count"] * (live // c["rows"] + 1)
        return {"bytes": 2 * page * c["pools"] * c["count"] + 4 * (3 * entries + 2 * c["n_pages"]), "flops": 0}
    moved = int(live * (1 - live / c["n_pages"]))
    return {"bytes": 2 * page * c["pools"] * moved + 4 * (4 * c["n_pages"] + 2 * live), "flops": 0}


# ---------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return {"attn": exact_attn, "append": exact_append, "rope": exact_rope, "fork": exact_fork, "compact": exact_compact}[case["op"]](case, s)


def exact_attn(c, s):
    """Sequence by sequence and KV head by KV head, from the pages that hold its keys."""
    new, ctx = lengths(c)
    if work(c)["flops"] > 4e12:
        return None
    G, ps, D = c["Hq"] // c["Hkv"], c["ps"], c["D"]
    out = torch.zeros((c["Hq"], s["total"], D), dtype=F64, device="cuda")
    out_lse = torch.zeros((c["Hq"], s["total"]), dtype=F64, device="cuda")
    first = 0
    for b, (n, x) in enumerate(zip(new, ctx)):
        row = s["table"][b, :-(-(n + x) // ps)].cpu().tolist()
        held = [(i, p) for i, p in enumerate(row) if p >= 0]
        if held:
            where = torch.cat([torch.arange(i * ps, i * ps + ps) for i, _ in held])
            pick = (where < n + x).nonzero()[:, 0].cuda()
            where = where.cuda()[pick]
            ids = torch.tensor([p for _, p in held], device="cuda")
            for h in range(c["Hkv"]):
                k = s["k_pages"][ids, h].reshape(-1, D)[pick].double()
                v = s["v_pages"][ids, h].reshape(-1, D)[pick].double()
                for lo in range(0, n, 256):
                    hi = min(n, lo + 256)
                    z = s["q"][h * G:(h + 1) * G, first + lo:first + hi].double() @ k.T / math.sqrt(D)
                    if c["causal"]:
                        last = x + torch.arange(lo, hi, device="cuda")
                        z = torch.where(where > last[:, None], -math.inf, z)
                    lse = torch.logsumexp(z, -1)
                    w = torch.exp(z - torch.where(lse == -math.inf, 0.0, lse)[..., None])
                    out[h * G:(h + 1) * G, first + lo:first + hi] = w @ v
                    out_lse[h * G:(h + 1) * G, first + lo:first + hi] = lse
        else:
            out_lse[:, first:first + n] = -math.inf
        first += n
    return out, out_lse


def turned(x, pos, c, inverse):
    """x [H, n, D] as complex pairs times exp(i angle), pos [3, n]."""
    half = c["D"] // 2
    z = x.double()
    re, im = (z[..., 0::2], z[..., 1::2]) if c["interleaved"] else (z[..., :half], z[..., half:])
    axis = torch.tensor(axis_of_pairs(c["D"]), device="cuda")
    i = torch.arange(half, device="cuda", dtype=F64)
    angle = pos.double().T[:, axis] * torch.pow(torch.tensor(10000.0, dtype=F64, device="cuda"), -2.0 * i / c["D"])
    w = torch.complex(re, im) * torch.polar(torch.ones_like(angle), -angle if inverse else angle)
    y = torch.empty_like(z)
    if c["interleaved"]:
        y[..., 0::2], y[..., 1::2] = w.real, w.imag
    else:
        y[..., :half], y[..., half:] = w.real, w.imag
    return y


def exact_rope(c, s):
    made = []
    for n, inverse in (("q", False), ("k", False), ("dq", True), ("dk", True)):
        made.append(torch.stack([turned(s[n][b], s["pos"][:, b], c, inverse) for b in range(c["B"])]))
    return (made[0], made[1]), (made[2], made[3])


def exact_append(c, s):
    new, ctx = lengths(c)
    k, q = turned(s["k"], s["pos"], c, False), turned(s["q"], s["pos"], c, False)
    k_pages, v_pages = s["k_pages"].double(), s["v_pages"].double()
    table, ps, first = s["table"].cpu(), c["ps"], 0
    for b, (n, x) in enumerate(zip(new, ctx)):
        done = 0
        while done < n:  # page by page
            at = x + done
            m = min(n - done, ps - at % ps)
            p = int(table[b, at // ps])
            for pool, fresh in ((k_pages, k), (v_pages, s["v"].double())):
                pool[p, :, at % ps:at % ps + m] = fresh[:, first + done:first + done + m]
            done += m
        first += n
    return q, k_pages, v_pages


def lowest_free(refs):
    for p, r in enumerate(refs):
        if r == 0:
            return p
    raise ValueError("no free page")


def exact_fork(c, s):
    """The tables page by page on the host; the children are free at the start."""
    table, lens, refs, ps = s["table"].cpu().tolist(), s["lens"].cpu().tolist(), s["refs"].cpu().tolist(), c["ps"]
    pool = s["pool"].double()
    for a, b in zip(s["src"].tolist(), s["dst"].tolist()):
        for i in range(lens[a] // ps):
            table[b][i] = table[a][i]
            refs[table[a][i]] += 1
        if lens[a] % ps:
            p = lowest_free(refs)
            refs[p] = 1
            table[b][lens[a] // ps] = p
            pool[:, p] = pool[:, table[a][lens[a] // ps]]
        lens[b] = lens[a]
    for b, n in enumerate(s["n_new"].cpu().tolist()):
        for i in range(-(-lens[b] // ps), -(-(lens[b] + n) // ps)):
            table[b][i] = lowest_free(refs)
            refs[table[b][i]] = 1
        lens[b] += n
    whole = lambda x: torch.tensor(x, dtype=I32, device="cuda")  # noqa: E731
    return pool, whole(table), whole(lens), whole(refs), torch.zeros_like(s["status"]), torch.zeros_like(s["status_new"])


def exact_compact(c, s):
    table, refs = s["table"].cpu().tolist(), s["refs"].cpu().tolist()
    pool = s["pool"].double()
    n_live = sum(r > 0 for r in refs)
    moves = dict(zip([p for p in range(n_live, len(refs)) if refs[p] > 0], [p for p in range(n_live) if refs[p] == 0]))
    for a, b in moves.items():
        pool[:, b] = pool[:, a]
        refs[b], refs[a] = refs[a], 0
    table = [[moves.get(p, p) for p in row] for row in table]
    whole = lambda x: torch.tensor(x, dtype=I32, device="cuda")  # noqa: E731
    return pool, whole(table), whole(refs), whole([n_live])

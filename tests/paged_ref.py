"""64-bit definitions of the serving-side operators and the error bounds of their kernels, for the tests.

Rounding to a type is off by at most half a step, relative to the value: bf16 2^-8, fp32 2^-24.
"""
import math

import torch

BF16_HALF, F32_HALF = 2.0 ** -8, 2.0 ** -24


def attention(q, k_pages, v_pages, table, kv_lens, cu, causal, scale):
    """O, lse in fp64 and their bounds: [Hq, total, D] / [Hq, total], rows of no sequence NaN.

    With p the exact softmax, s the scores, n the keys of a row:
      * a score's fp32 dot product is off by at most (D + 2) 2^-24 scale sum_d |q_d k_d| =: ds, which moves every p by
        a factor 1 + ds, numerator and normaliser;
      * 2^x on the special-function unit and the fp32 exponent argument: 2^-22 and |x| 2^-24 with |x| below
        log2(e) max |s - m|; keys further than 40 below the maximum add less than e^-40 n of the sum, so |x| <= 64: 2^-18;
      * sums of n terms in fp32, in tiles and over partials: n 2^-24, twice (numerator and normaliser), and 2^-20 for
        the merge weights and divisions;
      * P is rounded to bf16 before P V: 2^-8 on each term of the numerator only;
      * O is rounded to bf16 once: 2^-8 |O|."""
    Hq, total, D = q.shape
    n_pages, Hkv, ps, _ = k_pages.shape
    G = Hq // Hkv
    o = torch.full((Hq, total, D), math.nan, dtype=torch.float64)
    o_tol = torch.zeros_like(o)
    lse = torch.full((Hq, total), math.nan, dtype=torch.float64)
    lse_tol = torch.zeros_like(lse)
    q, k_pages, v_pages = q.double().cpu(), k_pages.cpu(), v_pages.cpu()
    table, kv_lens, cu = table.cpu(), kv_lens.cpu().tolist(), cu.cpu().tolist()
    for b, kv in enumerate(kv_lens):
        a, e = cu[b], cu[b + 1]
        if e <= a:
            continue
        kv = max(0, min(kv, table.shape[1] * ps))
        keys = [(i, int(table[b, i // ps]), i % ps) for i in range(kv) if 0 <= int(table[b, i // ps]) < n_pages]
        at = torch.tensor([x[0] for x in keys], dtype=torch.long)
        pg, sl = torch.tensor([x[1] for x in keys], dtype=torch.long), torch.tensor([x[2] for x in keys], dtype=torch.long)
        for h in range(Hq):
            k = k_pages[pg, h // G, sl].double().reshape(-1, D)
            v = v_pages[pg, h // G, sl].double().reshape(-1, D)
            x = q[h, a:e]
            s = x @ k.T * scale
            ds = (D + 2) * F32_HALF * scale * (x.abs() @ k.abs().T)
            if causal:
                last = kv - (e - a) + torch.arange(e - a)
                s = torch.where(at[None, :] > last[:, None], -math.inf, s)
            n = max(1, len(keys))
            z = torch.logsumexp(s, -1) if keys else torch.full((e - a,), -math.inf, dtype=torch.float64)
            w = torch.exp(s - torch.where(z == -math.inf, 0.0, z)[:, None])
            out = w @ v
            rel = 2 * ds.amax(-1) if keys else torch.zeros(e - a, dtype=torch.float64)
            rel = rel + 2.0 ** -17 + 2 * n * F32_HALF + 2.0 ** -20
            o[h, a:e], lse[h, a:e] = out, z
            o_tol[h, a:e] = (w @ v.abs()) * (rel[:, None] + BF16_HALF) * (1 + BF16_HALF) + BF16_HALF * out.abs() + 1e-30
            # lse = ln2 (m + log2 l): the relative error of l, and a few fp32 roundings of the result
            lse_tol[h, a:e] = rel + 8 * F32_HALF * torch.where(z == -math.inf, 0.0, z).abs() + 2.0 ** -20
    return o, o_tol, lse, lse_tol


def check_attention(got, ref, rows=None):
    """Elementwise within the bounds; rows that see no key exactly 0 / -inf."""
    (o, lse), (o_ref, o_tol, l_ref, l_tol) = got, ref
    o, lse = o.double().cpu(), lse.double().cpu()
    mine = ~torch.isnan(l_ref)
    if rows is not None:
        mine = mine & rows
    empty = mine & (l_ref == -math.inf)
    assert torch.equal(torch.isneginf(lse) & mine, empty), "rows that see no key"
    assert (o[empty] == 0).all()
    full = mine & ~empty
    assert torch.isfinite(o[full]).all() and torch.isfinite(lse[full]).all()
    worst_o = ((o - o_ref).abs() / o_tol)[full].max().item() if full.any() else 0.0
    worst_l = ((lse - l_ref).abs() / l_tol)[full].max().item() if full.any() else 0.0
    assert worst_o <= 1.0, f"O at {worst_o:.2f}x its bound"
    assert worst_l <= 1.0, f"lse at {worst_l:.2f}x its bound"


def rotate(x, pos, inv_freq, axes, interleaved, inverse=False):
    """x [B, H, S, D] turned by pos [n_axes, B, S] in fp64, and the bound of the kernel's result."""
    D = x.shape[-1]
    axes = [int(a) for a in axes]
    f = torch.as_tensor([float(v) if a >= 0 else 0.0 for v, a in zip(inv_freq, axes)], dtype=torch.float64)
    turned = torch.stack([pos[max(a, 0)] for a in axes], -1).double().cpu()[:, None]  # [B, 1, S, D/2]
    angle = turned * f * (-1.0 if inverse else 1.0)
    c, s = angle.cos(), angle.sin()
    z = x.double().cpu()
    a, b = (z[..., 0::2], z[..., 1::2]) if interleaved else (z[..., :D // 2], z[..., D // 2:])
    y1, y2 = a * c - b * s, a * s + b * c
    # The angle: turns as a float, 2^-24 of at most half a turn, in radians pi 2^-24 < 2^-22; the double frequency,
    # here and in the kernel, 2^-52 of the angle; sincospif within 2 units, 2^-23; two fp32 roundings of each product.
    err = (a.abs() + b.abs()) * (2.0 ** -22 + 2.0 ** -23 + 2 * F32_HALF + 4 * angle.abs() * 2.0 ** -52)
    half = BF16_HALF if x.dtype == torch.bfloat16 else F32_HALF
    t1, t2 = err + half * (y1.abs() + err), err + half * (y2.abs() + err)
    y, tol = torch.empty_like(z), torch.empty_like(z)
    if interleaved:
        y[..., 0::2], y[..., 1::2], tol[..., 0::2], tol[..., 1::2] = y1, y2, t1, t2
    else:
        y[..., :D // 2], y[..., D // 2:], tol[..., :D // 2], tol[..., D // 2:] = y1, y2, t1, t2
    return y, tol + 1e-30


def within(got, ref, tol):
    worst = ((got.double().cpu() - ref).abs() / tol).max().item()
    assert worst <= 1.0, f"{worst:.2f}x the bound"


class Tables:
    """Host model of the page tables: the definition of reserve, fork, free and compact."""

    def __init__(self, table, lens, refs, ps):
        self.table = [list(map(int, r)) for r in table]
        self.lens, self.refs, self.ps = list(map(int, lens)), list(map(int, refs)), ps

    def free_list(self):
        return [p for p, r in enumerate(self.refs) if r == 0]

    def reserve(self, n_new):
        """Rows are served in order while the free pages last; a row's pages count even if it is not served."""
        free, at, status = self.free_list(), 0, []
        for b, n in enumerate(n_new):
            n, ln, W = max(n, 0), self.lens[b], len(self.table[b])
            if ln + n > W * self.ps:
                status.append(2)
                continue
            have, want = -(-ln // self.ps), -(-(ln + n) // self.ps)
            at += want - have
            if want > have and at > len(free):
                status.append(1)
                continue
            for i in range(have, want):
                self.table[b][i] = free[at - want + i]
                self.refs[self.table[b][i]] = 1
            self.lens[b] = ln + n
            status.append(0)
        return status

    def fork(self, src, dst):
        free, at, status, copies = self.free_list(), 0, [], []
        for a, b in zip(src, dst):
            if self.lens[b]:
                status.append(3)
                continue
            whole, part = divmod(self.lens[a], self.ps)
            if part:
                at += 1
                if at > len(free):
                    status.append(1)
                    continue
            row = self.table[a][:whole] + [-1] * (len(self.table[b]) - whole)
            for p in row[:whole]:
                if 0 <= p < len(self.refs):
                    self.refs[p] += 1
            if part:
                row[whole] = free[at - 1]
                self.refs[row[whole]] = 1
                copies.append((self.table[a][whole], row[whole]))
            self.table[b], self.lens[b] = row, self.lens[a]
            status.append(0)
        return status, copies

    def free(self, rows):
        for b in rows:
            for p in self.table[b]:
                if 0 <= p < len(self.refs):
                    self.refs[p] -= 1
            self.table[b] = [-1] * len(self.table[b])
            self.lens[b] = 0

    def compact(self):
        n = sum(r > 0 for r in self.refs)
        moves = list(zip([p for p in range(n, len(self.refs)) if self.refs[p] > 0],
                         [p for p in range(n) if self.refs[p] <= 0]))
        to = dict(moves)
        for a, b in moves:
            self.refs[b], self.refs[a] = self.refs[a], 0
        self.table = [[to.get(p, p) for p in row] for row in self.table]
        return n, moves

"""Bounds of the attention over the 8-bit cache that follow its weights one by one (drafts_ref.attention grants a floor
that grows with the keys).

Narrow form (at most 64 rows a KV head). A weight with its value's scale, W = 2^(s + e), against a reference R with W <= 2^4 R,
is rounded to fp16 (2^-11 of itself) and then held as three e5m2 numbers: upper byte, upper byte of the rest, the rest of that
to nearest times 2^4. Each takes three bits, so 2^-9 is off at most; below, half of e5m2's smallest step, 2^-17 / 2^4, where R is
2^11: 2^-32 R. R is no more than the row's largest W -- or, of values that differ by more than 2^44, 2^(E - 44) times its largest
2^s, E the largest exponent of the values that its sequence's rows see.
Wide form. Weights 2^s are rounded to fp16 (2^-11), or by half of its smallest step, 2^-25, where a tile of 128 keys whose weights
sum to less than 2^-7 gets a new reference, against which its largest weight is 2^5: 2^-18 of its sum. In the first tile the
largest is 2^13: 2^-38 of it. Values are codes times factors, in a unit U of at most 2^-2 of the tile's largest scale: exact
while the factor is 2^-15 or more (a code's last bit is 2^-9), so down to 2^-17 of the largest scale; then off by half a step,
2^-25 U, 2^-27 of the largest scale; and lost where the factor is below fp16's last step, 2^-24: below 2^-26 of that scale. (Units fall 2^-40 behind
the largest at most, and that is 2^-2 of a scale: 2^-60 of the largest one of all; references as far as l stays below 2^57: 2^-70 of
all.)
Both. Scores as in drafts_ref.attention; keys of the wide form, in a unit of 2^-7 of the tile's largest scale, are exact down to
2^-22 of that, then off by 2^-32 of it, and lost below 2^-31."""
import math

import torch

from tests.paged_ref import BF16_HALF, F32_HALF

U8 = torch.uint8


def exponents(scales):
    return scales.view(U8).double() - 127


def attention(q, k, v, ek, ev, codes, seen, scale, wide, at=None):
    """One sequence and KV head, on any device, in 64 bits: q [R, D], values k, v [n, D], exponents ek, ev [n], codes of v [n, D],
    seen [R, n] -> O, its bound, lse, its bound, and of O's norm what the floors of the wide form's first tile and of its values can take. at [n]: the keys' places in the sequence (0 .. n - 1 if not given)."""
    q, k, v, ek, ev, codes = (x.double() for x in (q, k, v, ek, ev, codes))
    n, D = k.shape
    tile = (torch.arange(n, device=k.device) if at is None else at) // 128
    n_tiles = int(tile.max()) + 1 if n else 0
    most = lambda x: torch.full((n_tiles,), -1e4, dtype=torch.float64, device=x.device).scatter_reduce_(0, tile, x, "amax")[tile]  # noqa: E731
    s = q @ k.T * scale
    ds = 1.25 * (2 * D + 2) * F32_HALF * scale * (q.abs() @ k.abs().T)
    ds = ds + 2.0 ** -17 * scale * q.abs().amax(-1, keepdim=True) * k.abs().sum(-1)
    if wide:
        far = torch.where(ek < most(ek) - 22, 2.0 ** (most(ek) - 32), 0.0)
        ds = ds + scale * q.abs().sum(-1, keepdim=True) * far
        ds = ds + scale * (q.abs() @ torch.where((ek < most(ek) - 31)[:, None], k.abs(), 0.0).T)
    s = torch.where(seen, s, -math.inf)
    some = seen.any(-1)
    z = torch.where(some, torch.logsumexp(s, -1), -math.inf)
    z0 = torch.where(some, z, 0.0)
    w = torch.exp(s - z0[:, None])
    o = w @ v
    rel = 2 * torch.where(seen, ds, 0.0).amax(-1) + 2.0 ** -17 + 2 * n * F32_HALF + 2.0 ** -20
    tol = (w @ v.abs()) * rel[:, None] * (1 + BF16_HALF)
    taken = torch.zeros_like(z)
    if wide:
        tol = tol + (w @ v.abs()) * (2.0 ** -11 * (1 + BF16_HALF))
        sums = torch.zeros((q.shape[0], n_tiles), dtype=torch.float64, device=k.device).index_add_(1, tile, w)
        sizes = torch.zeros((n_tiles, D), dtype=torch.float64, device=k.device)
        # (a key that a row does not see has no weight; counting its value only widens the bound)
        sizes.index_add_(0, tile, v.abs())
        floor = 2.0 ** -18 * sums
        floor[:, 0] = 2.0 ** -38 * torch.where(tile == 0, w, 0.0).amax(-1)
        beside = torch.where(tile == 0, torch.minimum(w, floor[:, :1]), 0.0)
        taken = (beside @ v.abs()).norm(dim=-1) / o.norm(dim=-1).clamp(min=1e-300)
        floor = floor + 2.0 ** -70
        tol = tol + floor @ sizes
        small = torch.where(ev < most(ev) - 17, 2.0 ** (most(ev) - 27), 0.0)[:, None] + (2.0 ** (ev.amax() - 60) if n else 0.0)
        lost = torch.where((ev < most(ev) - 26)[:, None], v.abs(), small)
        tol = tol + w @ lost
        taken = taken + (w @ lost).norm(dim=-1) / o.norm(dim=-1).clamp(min=1e-300)
    else:
        tol = tol + (w @ v.abs()) * ((2.0 ** -9 + 2.0 ** -11) * (1 + BF16_HALF))
        top_e = ev[seen.any(0)].amax() if bool(seen.any()) else 0.0
        unit = torch.maximum((w * 2.0 ** ev).amax(-1), w.amax(-1) * 2.0 ** (top_e - 44))
        tol = tol + 2.0 ** -32 * (1 + 2.0 ** -3) * unit[:, None] * (seen.double() @ codes.abs())
    tol = tol + BF16_HALF * o.abs() + 1e-30
    return o, tol, z, rel + 8 * F32_HALF * z0.abs() + 2.0 ** -20, taken

"""The serving side: attention over a paged K/V cache (bf16 or e4m3), rotary
positions with several axes, appends to the cache and the management of its pages,
drafts and their trees, over the C ABI of include/seqattn_paged.h.

    plan = RopePlan(128, sections=(16, 24, 24))              # time, height, width
    q, k = rope_axes(q, k, positions, *plan)                 # training; gradients: rope_axes_bwd
    cache = PagedCache(n_pages=4096, Hkv=4, D=128, rows=64, max_pages=512, page_size=16, plan=plan)
    cache.reserve(n_new)                                      # room for the next tokens of every row
    o, lse = cache.step(0, q, k, v, cu_seqlens, positions)    # append, then attend (layer 0)
    cache.fork([0, 0], [8, 9]); cache.free([3]); cache.compact()

    cache = PagedCache(..., dtype=torch.float8_e4m3fn)        # half the bytes: codes and a scale per key and value
    tree, depths = draft_tree(parents, cu_seqlens)            # drafts that branch: masks for every layer
    o, lse = cache.step(0, q, k, v, cu_seqlens, positions, tree=tree)
    path, n_keep, last = draft_accept(parents, cu_seqlens, tokens, choices, tree=tree)
    status = cache.keep(cu_seqlens, path, n_keep)             # the rejected drafts leave the cache

New tokens are packed: [H, total, D] tensors (any strides with D contiguous and
16-byte multiples, so a transposed [total, H, D] projection goes in without a
copy), sequence b in rows cu_seqlens[b] .. cu_seqlens[b + 1]. Page tables,
lengths, reference counts and cu_seqlens are int32 CUDA tensors, read on the
device: a captured call follows their contents. Lists of rows or pages are host
sequences (or CPU int32 tensors), checked before anything is launched.
"""
from __future__ import annotations

import functools
import math
import struct

import torch

from . import ATTN_BF16, ATTN_F32, _check, _require
from ._lib import lib

PAGED_NO_PAGES, PAGED_TOO_LONG, PAGED_IN_USE = 1, 2, 3
PAGED_BAD_PATH, PAGED_SHARED, PAGED_REFUSED = 4, 5, 6
DRAFT_MAX_WORDS = 4
_BF16, _F32, _I32, _I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64
_E4M3, _E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
# paged_cache and rope_rows of include/seqattn_paged.h, packed (cheaper per call than ctypes structures)
_CACHE = struct.Struct("@PPqPqPPiiiiii")
_ROWS = struct.Struct("@PPqqqqqqi4x")
_SCALES = struct.Struct("@PPq")
_POOL = struct.Struct("@Pqqqi4x")  # paged_pool


def _call(fn, what: str, dev: int, *args) -> None:
    """fn(*args, stream) with device `dev` current (the kernels launch there), on its current stream."""
    if torch._C._cuda_getDevice() == dev:
        st = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        with torch.cuda.device(dev):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    if st != 0:
        _check(st, what)


def _one_device(what: str, *tensors) -> int:
    dev = tensors[0].get_device()
    for t in tensors:
        if dev < 0 or t.get_device() != dev:
            raise ValueError(f"{what}: all tensors must be on one CUDA device")
    return dev


def _host_ints(x, what: str) -> torch.Tensor:
    """A host list of ints as a contiguous int32 CPU tensor."""
    if not isinstance(x, torch.Tensor):
        x = torch.tensor([int(v) for v in x], dtype=_I32)
    if x.is_cuda or x.dtype != _I32 or x.dim() != 1:
        raise ValueError(f"{what} must be host ints (or int32 CPU)")
    return x if x.is_contiguous() else x.contiguous()


def _ints(t: torch.Tensor, n: int, what: str) -> None:
    if t.dtype != _I32 or t.dim() != 1 or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous int32 [{n}]")


def _tables(page_table: torch.Tensor, kv_lens=None, page_refs=None):
    """(rows, columns, row stride) of the page table."""
    if page_table.dim() != 2 or page_table.dtype != _I32:
        raise ValueError("page_table must be int32 [B, max_pages]")
    (B, W), (sb, sw) = page_table.shape, page_table.stride()
    if (W > 1 and sw != 1) or (B > 1 and sb < W):
        raise ValueError("page_table must have contiguous rows that do not overlap")
    if kv_lens is not None:
        _ints(kv_lens, B, "kv_lens")
    if page_refs is not None and (page_refs.dtype != _I32 or page_refs.dim() != 1 or not page_refs.is_contiguous()
                                  or page_refs.numel() == 0):
        raise ValueError("page_refs must be contiguous int32 [n_pages]")
    return B, W, sb if B > 1 else W


def _guard(guard, B: int, used: list):
    """The guard's address (it joins `used`), or None."""
    if guard is None:
        return None
    if guard.dtype != _I32 or guard.shape != (4, B) or not guard.is_contiguous():
        raise ValueError(f"guard must be contiguous int32 [4, {B}]")
    used.append(guard)
    return guard.data_ptr()


def _distinct_memory(t: torch.Tensor, what: str) -> None:
    """Every dimension longer than one has a non-zero stride (no expanded output)."""
    if 0 in t.stride() and any(n > 1 and s == 0 for n, s in zip(t.shape, t.stride())):
        raise ValueError(f"{what} must not be expanded")


def _packed(t: torch.Tensor, total: int, D: int, what: str):
    """Strides of bf16 rows [H, total, D] with D contiguous."""
    if t.dim() != 3 or t.dtype != _BF16 or t.shape[1] != total or t.shape[2] != D or t.stride(2) != 1:
        raise ValueError(f"{what} must be bf16 [H, {total}, {D}] with D contiguous")
    return t.stride()


def _cache_view(k_pages, v_pages, page_table, kv_lens, cu_seqlens, k_scales=None, v_scales=None):
    """paged_cache as bytes, its device, and (B, Hkv, D)."""
    if k_pages.dim() != 4 or v_pages.shape != k_pages.shape:
        raise ValueError("pools must be [n_pages, Hkv, page_size, D]")
    n_pages, Hkv, ps, D = k_pages.shape
    sk, sv = k_pages.stride(), v_pages.stride()
    dtype = _BF16 if k_scales is None and v_scales is None else _E4M3
    if (k_pages.dtype != dtype or v_pages.dtype != dtype or sk[3] != 1 or sv[3] != 1
            or (ps > 1 and (sk[2] != D or sv[2] != D)) or (Hkv > 1 and (sk[1] != ps * D or sv[1] != ps * D))):
        raise ValueError("pools must be bf16 (or, with scales, float8_e4m3fn) with contiguous pages")
    if n_pages > 1 and sv[0] != sk[0]:
        raise ValueError("the K and V pools must share their page stride")
    B, W, row = _tables(page_table, kv_lens)
    _ints(cu_seqlens, B + 1, "cu_seqlens")
    dev = _one_device("the cache (CUDA tensors)", k_pages, v_pages, page_table, kv_lens, cu_seqlens)
    return _CACHE.pack(k_pages.data_ptr(), v_pages.data_ptr(), sk[0] if n_pages > 1 else Hkv * ps * D,
                       page_table.data_ptr(), row, kv_lens.data_ptr(), cu_seqlens.data_ptr(), B, n_pages, ps, W, Hkv,
                       D), dev, B, Hkv, D


def _scales_view(k_pages, k_scales, v_scales, used: list):
    """paged_scales as bytes (the scales join `used`), or None of a bf16 cache."""
    if k_scales is None and v_scales is None:
        return None
    if k_scales is None or v_scales is None:
        raise ValueError("k_scales and v_scales go together")
    n_pages, Hkv, ps, _ = k_pages.shape
    sk, sv = k_scales.stride(), v_scales.stride()
    for t, s in ((k_scales, sk), (v_scales, sv)):
        if (t.dtype != _E8M0 or t.shape != (n_pages, Hkv, ps) or (ps > 1 and s[2] != 1) or (Hkv > 1 and s[1] != ps)
                or (n_pages > 1 and s[0] != sk[0])):
            raise ValueError(f"scales must be float8_e8m0fnu [{n_pages}, {Hkv}, {ps}] with contiguous pages of one stride")
    used += (k_scales, v_scales)
    return _SCALES.pack(k_scales.data_ptr(), v_scales.data_ptr(), sk[0] if n_pages > 1 else Hkv * ps)


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(Hq: int, Hkv: int, total_q: int, D: int) -> int:
    """The library's answer for these sizes (a call of its own otherwise)."""
    return int(lib.attn_paged_workspace_bytes(Hq, Hkv, total_q, D))


def attn_paged_workspace_bytes(Hq: int, Hkv: int, total_q: int, D: int) -> int:
    """Device workspace bytes attn_paged needs."""
    n = _workspace_bytes(Hq, Hkv, total_q, D)
    _require(n > 0, "invalid sizes")
    return n


def attn_paged(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor,
               kv_lens: torch.Tensor, cu_seqlens: torch.Tensor, causal: bool = True, scale: float | None = None,
               out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None, tree: torch.Tensor | None = None,
               k_scales: torch.Tensor | None = None, v_scales: torch.Tensor | None = None):
    """Attention of the packed new tokens q bf16 [Hq,total_q,D] over a paged cache.

    k_pages / v_pages bf16 [n_pages,Hkv,page_size,D]; page_table int32
    [B,max_pages] (an entry that is no page: its keys are not seen); kv_lens int32
    [B], the new tokens included (their keys are the last ones); cu_seqlens int32
    [B+1]. Under the causal mask token t of a sequence sees the keys up to its
    own. Returns (O bf16 [Hq,total_q,D], lse fp32 [Hq,total_q]); rows that see no
    key get O = 0, lse = -inf, rows of no sequence keep what out / lse held
    (unspecified where they are made here). workspace: a uint8 CUDA tensor of
    attn_paged_workspace_bytes(...), for one call at a time (made per call when
    not given).

    tree: masks int64 [total_q, words] (draft_tree), words at most 4: a token of a
    sequence of at most 64 * words new ones sees the cached keys and, of the new ones,
    those whose bits are set in its mask; longer sequences are causal as without.
    k_scales / v_scales float8_e8m0fnu [n_pages,Hkv,page_size]: the pools are
    float8_e4m3fn, an element is code * scale."""
    if q.dim() != 3:
        raise ValueError("expected q [Hq, total_q, D]")
    Hq, total, D = q.shape
    view, dev, B, Hkv, d = _cache_view(k_pages, v_pages, page_table, kv_lens, cu_seqlens, k_scales, v_scales)
    if d != D or Hkv == 0 or Hq % Hkv != 0:
        raise ValueError("q must have the cache's D and a multiple of its heads")
    sq = _packed(q, total, D, "q")
    where, used = q.device, [k_pages, q]
    scales = _scales_view(k_pages, k_scales, v_scales, used)
    masks, words = None, 0
    if tree is not None:
        if tree.dtype != _I64 or tree.dim() != 2 or tree.shape[0] != total or not tree.is_contiguous():
            raise ValueError(f"tree must be contiguous int64 [{total}, words]")
        masks, words = tree.data_ptr(), tree.shape[1]
        _require(1 <= words <= DRAFT_MAX_WORDS, "a tree's masks have one to four words")
        _require(causal, "a tree says itself what its tokens see: causal=False is of no use with it")
        used.append(tree)
    if out is None:
        out, so = torch.empty((Hq, total, D), dtype=_BF16, device=where), (total * D, D)
    else:
        _distinct_memory(out, "out")
        so = _packed(out, total, D, "out")
        if out.shape[0] != Hq:
            raise ValueError("bad out")
        used.append(out)
    if lse is None:
        lse = torch.empty((Hq, total), dtype=_F32, device=where)
    else:
        if lse.dtype != _F32 or lse.shape != (Hq, total) or not lse.is_contiguous():
            raise ValueError("bad lse")
        used.append(lse)
    if total == 0 or B == 0:
        return out, lse
    need = _workspace_bytes(Hq, Hkv, total, D)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=where)
    else:
        if workspace.dtype != torch.uint8 or not workspace.is_contiguous() or workspace.numel() < need:
            raise ValueError("workspace must be a contiguous uint8 tensor of attn_paged_workspace_bytes(...) bytes")
        used.append(workspace)
    _one_device("attn_paged", *used)
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    to = out.data_ptr(), so[0], so[1], lse.data_ptr(), workspace.data_ptr(), workspace.numel(), Hq, total
    if scales is not None:
        _call(lib.attn_paged_e4m3, "attn_paged_e4m3", dev, q.data_ptr(), sq[0], sq[1], view, scales, *to,
              1 if causal else 0, masks, words, scale)
    elif tree is not None:
        _call(lib.attn_paged_tree, "attn_paged_tree", dev, q.data_ptr(), sq[0], sq[1], view, *to, masks, words, scale)
    else:
        _call(lib.attn_paged, "attn_paged", dev, q.data_ptr(), sq[0], sq[1], view, *to, 1 if causal else 0, scale)
    return out, lse


class RopePlan:
    """The frequencies and axes of a rotary embedding: ``inv_freq`` (float64) and
    ``axes`` (int32), CPU tensors of D / 2; unpacks as the two. Pair i turns
    by position[axes[i]] * base^(-2 i / D); sections gives the number of pairs of
    each axis in turn (their sum may fall short of D / 2: the last pairs are not
    turned). shared=False: each axis has its own ladder over its section."""

    def __init__(self, D: int, sections=None, base: float = 10000.0, shared: bool = True):
        sections = (D // 2,) if sections is None else tuple(int(s) for s in sections)
        _require(min(sections) >= 0 and sum(sections) <= D // 2, "sections must fit in D / 2 pairs")
        freq, axes = [], []
        for a, n in enumerate(sections):
            for i in range(n):
                freq.append(base ** (-2.0 * len(freq) / D) if shared else base ** (-i / n))
                axes.append(a)
        rest = D // 2 - len(axes)
        self.inv_freq = torch.tensor(freq + [0.0] * rest, dtype=torch.float64)
        self.axes = torch.tensor(axes + [-1] * rest, dtype=_I32)

    def __iter__(self):
        return iter((self.inv_freq, self.axes))


def _plan(inv_freq, axes, D: int):
    if not isinstance(inv_freq, torch.Tensor):
        inv_freq = torch.tensor([float(f) for f in inv_freq], dtype=torch.float64)
    axes = _host_ints(axes, "axes")
    if inv_freq.is_cuda or inv_freq.dtype != torch.float64 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise ValueError("inv_freq must be host floats (or float64 CPU)")
    if inv_freq.numel() != D // 2 or axes.numel() != D // 2:
        raise ValueError("inv_freq and axes need D / 2 entries")
    return inv_freq, axes


def _rope(q, k, positions, inv_freq, axes, interleaved, inverse, out_q, out_k):
    first = k if q is None else q
    if first is None:
        raise ValueError("q or k is needed")
    if first.dim() != 4:
        raise ValueError("rows must be [B, H, S, D]")
    B, _, S, D = first.shape
    dtype = first.dtype
    if dtype != _BF16 and dtype != _F32:
        raise ValueError("rows must be bf16 or fp32")
    views, outs, used = [None, None], [None, None], [positions]
    for i, (t, o) in enumerate(((q, out_q), (k, out_k))):
        if t is None:
            continue
        if o is None:
            o = torch.empty(t.shape, dtype=dtype, device=t.device)
        else:
            _distinct_memory(o, "out")
        st, so, shape = t.stride(), o.stride(), t.shape
        if (len(shape) != 4 or o.shape != shape or shape[0] != B or shape[2] != S or shape[3] != D or t.dtype != dtype
                or o.dtype != dtype or st[3] != 1 or so[3] != 1):
            raise ValueError("rows must be [B, H, S, D] of one dtype with D contiguous")
        views[i] = _ROWS.pack(t.data_ptr(), o.data_ptr(), st[0], st[1], st[2], so[0], so[1], so[2], shape[1])
        outs[i] = o
        used += (t, o)
    if positions.dim() != 3 or positions.dtype != _I32 or positions.shape[1] != B or positions.shape[2] != S:
        raise ValueError("positions must be int32 [n_axes, B, S]")
    sp = positions.stride()
    if S > 1 and sp[2] != 1:
        raise ValueError("positions must be contiguous along S")
    inv_freq, axes = _plan(inv_freq, axes, D)
    dev = _one_device("rope_axes", *used)
    _call(lib.rope_axes, "rope_axes", dev, views[0], views[1], positions.data_ptr(), sp[0], sp[1], positions.shape[0],
          inv_freq.data_ptr(), axes.data_ptr(), B, S, D, ATTN_F32 if dtype == _F32 else ATTN_BF16,
          1 if interleaved else 0, inverse)
    return outs[0], outs[1]


def rope_axes(q, k, positions: torch.Tensor, inv_freq, axes, interleaved: bool = False, out_q=None, out_k=None):
    """q [B,Hq,S,D] and k [B,Hkv,S,D] (bf16 or fp32, either may be None) turned by
    their positions: int32 [n_axes,B,S] (may be expanded along B). Pair i, i < D/2,
    turns by positions[axes[i]] * inv_freq[i]; it is the elements (i, i + D/2), or
    (2i, 2i+1) with interleaved. inv_freq / axes: host, D / 2 entries (RopePlan);
    axis -1: not turned. out_q / out_k may be q / k. Returns (q', k')."""
    return _rope(q, k, positions, inv_freq, axes, interleaved, 0, out_q, out_k)


def rope_axes_bwd(dq, dk, positions: torch.Tensor, inv_freq, axes, interleaved: bool = False, out_dq=None, out_dk=None):
    """Gradients of rope_axes: the output gradients turned back."""
    return _rope(dq, dk, positions, inv_freq, axes, interleaved, 1, out_dq, out_dk)


def paged_append(k: torch.Tensor, v: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor,
                 page_table: torch.Tensor, kv_lens: torch.Tensor, cu_seqlens: torch.Tensor, q=None, positions=None,
                 inv_freq=None, axes=None, interleaved: bool = False, out_q=None, guard: torch.Tensor | None = None,
                 k_scales: torch.Tensor | None = None, v_scales: torch.Tensor | None = None):
    """Writes the new tokens' k, v bf16 [Hkv,total,D] into the last slots of their
    sequences (kv_lens counts them already). With positions (int32
    [n_axes,total], inv_freq and axes as for rope_axes) k is turned on the way,
    and q [Hq,total,D] into out_q (may be q), which is returned. Tokens whose slot
    is on no page are dropped, and with a guard (that of the step's paged_reserve)
    those of rows that were refused room, which would lie over older keys; guard[3]
    then holds the lengths for the attention of the step, 0 for such a row. With
    k_scales / v_scales (as for attn_paged) the pools are float8_e4m3fn: k and v are
    rounded to code * scale, the scale the least power of two that holds the row (rows
    with an infinity lose their other elements; it is read as an infinity again)."""
    view, dev, B, Hkv, D = _cache_view(k_pages, v_pages, page_table, kv_lens, cu_seqlens, k_scales, v_scales)
    if k.dim() != 3:
        raise ValueError("expected k [Hkv, total, D]")
    if q is not None and positions is None:
        raise ValueError("q is turned by positions: pass them")
    total = k.shape[1]
    sk, sv = _packed(k, total, D, "k"), _packed(v, total, D, "v")
    if k.shape[0] != Hkv or v.shape[0] != Hkv:
        raise ValueError("k and v must have the cache's heads")
    used, vq = [k_pages, k, v], None
    scales = _scales_view(k_pages, k_scales, v_scales, used)
    if q is not None:
        sq = _packed(q, total, D, "q")
        if out_q is None:
            out_q = torch.empty(q.shape, dtype=_BF16, device=q.device)
        else:
            _distinct_memory(out_q, "out_q")
        so = _packed(out_q, total, D, "out_q")
        if out_q.shape != q.shape:
            raise ValueError("bad out_q")
        used += (q, out_q)
        vq = _ROWS.pack(q.data_ptr(), out_q.data_ptr(), 0, sq[0], sq[1], 0, so[0], so[1], q.shape[0])
    pos, pos_axis, n_axes, f, a = None, 0, 0, None, None
    if positions is not None:
        if positions.dim() != 2 or positions.dtype != _I32 or positions.shape[1] != total or (
                total > 1 and positions.stride(1) != 1):
            raise ValueError("positions must be int32 [n_axes, total]")
        inv_freq, axes = _plan(inv_freq, axes, D)
        pos, pos_axis, n_axes = positions.data_ptr(), positions.stride(0), positions.shape[0]
        f, a = inv_freq.data_ptr(), axes.data_ptr()
        used.append(positions)
    held = _guard(guard, B, used)
    _one_device("paged_append", *used)
    new = _ROWS.pack(k.data_ptr(), 0, 0, sk[0], sk[1], 0, 0, 0, Hkv), _ROWS.pack(v.data_ptr(), 0, 0, sv[0], sv[1], 0, 0, 0, Hkv)
    how = pos, pos_axis, n_axes, f, a, total, 1 if interleaved else 0, held
    if scales is None:
        _call(lib.paged_append_guarded, "paged_append", dev, vq, *new, view, *how)
    else:
        _call(lib.paged_append_e4m3, "paged_append_e4m3", dev, vq, *new, view, scales, *how)
    return out_q


def paged_read(k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor, kv_lens: torch.Tensor,
               cu_keys: torch.Tensor, total: int, first: torch.Tensor | None = None,
               k_scales: torch.Tensor | None = None, v_scales: torch.Tensor | None = None, out_k=None, out_v=None):
    """Keys and values out of the cache, bf16 [Hkv,total,D] each: rows cu_keys[b] ..
    cu_keys[b + 1] (int32 [B + 1], device) are the keys first[b] (int32 [B], device; 0
    when not given) on of sequence b. Keys that are not there come out as zeros; rows of
    no sequence keep what out_k / out_v held (unspecified where they are made here).
    With scales the pools are float8_e4m3fn (as for attn_paged); what comes out is
    exactly what they hold."""
    view, dev, B, Hkv, D = _cache_view(k_pages, v_pages, page_table, kv_lens, cu_keys, k_scales, v_scales)
    total, used = int(total), [k_pages]
    _require(total >= 0, "total must not be negative")
    scales = _scales_view(k_pages, k_scales, v_scales, used)
    outs = []
    for t, what in ((out_k, "out_k"), (out_v, "out_v")):
        if t is None:
            t = torch.empty((Hkv, total, D), dtype=_BF16, device=k_pages.device)
        else:
            _distinct_memory(t, what)
            used.append(t)
        st = _packed(t, total, D, what)
        _require(t.shape[0] == Hkv, f"{what} must have the cache's heads")
        outs.append((t, st))
    if first is not None:
        _ints(first, B, "first")
        used.append(first)
    _one_device("paged_read", *used)
    (k, sk), (v, sv) = outs
    _call(lib.paged_read, "paged_read", dev, view, scales, None if first is None else first.data_ptr(), k.data_ptr(), sk[0],
          sk[1], v.data_ptr(), sv[0], sv[1], total)
    return k, v


def _tokens(t: torch.Tensor, n: int, what: str, used: list) -> int:
    _ints(t, n, what)
    used.append(t)
    return t.data_ptr()


def draft_tree(parents: torch.Tensor, cu_seqlens: torch.Tensor, words: int = 1):
    """Masks int64 [total,words] and depths int32 [total] of drafts that branch, from
    their parents (int32 [total]: a token's parent as its number within its
    sequence's new tokens; negative, or not an earlier one: it follows the cached keys). Bit
    i of a mask is set for the token's ancestors and itself; depths counts the
    ancestors, so a token's position is kv_len - q_len + depth. A sequence of more than
    64 * words tokens is no tree: masks 0, depths 0, 1, 2, ... One call a step serves
    every layer."""
    used, total = [], parents.numel()
    at = _tokens(parents, total, "parents", used)
    _require(cu_seqlens.dim() == 1 and cu_seqlens.numel() >= 1, "cu_seqlens must be [B + 1]")
    cu = _tokens(cu_seqlens, cu_seqlens.numel(), "cu_seqlens", used)
    _require(1 <= words <= DRAFT_MAX_WORDS, "a tree's masks have one to four words")
    dev = _one_device("draft_tree", *used)
    masks = torch.empty((total, words), dtype=_I64, device=parents.device)
    depths = torch.empty(total, dtype=_I32, device=parents.device)
    _call(lib.draft_tree, "draft_tree", dev, at, cu, masks.data_ptr(), depths.data_ptr(), cu_seqlens.numel() - 1, total,
          int(words))
    return masks, depths


def draft_accept(parents: torch.Tensor, cu_seqlens: torch.Tensor, tokens: torch.Tensor, choices: torch.Tensor,
                 given: torch.Tensor | None = None, tree: torch.Tensor | None = None):
    """The drafts that the model confirms: from each sequence's given tokens (the first
    given[b], int32 [B] on the device; one when not given: the token that the step
    before chose) down the tree to the lowest child whose token is the model's choice
    behind its parent. tokens, choices int32 [total]: the token of each row, and what
    the model chose behind it. Returns (path int32 [total]: the kept tokens' numbers in
    rows cu_seqlens[b] .., then -1; n_keep int32 [B]; last int32 [B]: the choice
    behind the last kept token, -1 for a sequence without tokens). tree: the masks that the
    attention had (draft_tree). A sequence of more tokens than they have bits is a chain
    to it, and so here, whatever its parents; without tree, trees of any size are followed,
    those too whose choices the attention made as of a chain."""
    used, total = [], parents.numel()
    _require(cu_seqlens.dim() == 1 and cu_seqlens.numel() >= 1, "cu_seqlens must be [B + 1]")
    B = cu_seqlens.numel() - 1
    at = [_tokens(parents, total, "parents", used), _tokens(cu_seqlens, B + 1, "cu_seqlens", used),
          _tokens(tokens, total, "tokens", used), _tokens(choices, total, "choices", used),
          None if given is None else _tokens(given, B, "given", used)]
    words = 0
    if tree is not None:
        if tree.dtype != _I64 or tree.dim() != 2 or tree.shape[0] != total:
            raise ValueError(f"tree must be int64 [{total}, words]")
        words = tree.shape[1]
        _require(1 <= words <= DRAFT_MAX_WORDS, "a tree's masks have one to four words")
    dev = _one_device("draft_accept", *used)
    path = torch.empty(total, dtype=_I32, device=parents.device)
    n_keep, last = (torch.empty(B, dtype=_I32, device=parents.device) for _ in range(2))
    _call(lib.draft_accept_words, "draft_accept", dev, *at, path.data_ptr(), n_keep.data_ptr(), last.data_ptr(), B, total, words)
    return path, n_keep, last


def _slots(pools) -> tuple:
    """One pool or several; those of scales, [(L,) n_pages,Hkv,page_size], with a last dimension of one."""
    pools = (pools,) if isinstance(pools, torch.Tensor) else tuple(pools)
    return tuple(t.unsqueeze(-1) if t.dtype == _E8M0 else t for t in pools)


def _pools(pools, n_pages: int):
    """Pools [n_pages,Hkv,page_size,D] or [L,n_pages,Hkv,page_size,D] (one tensor or several) as paged_pool."""
    pools = _slots(pools)
    arr = b""
    for t in pools:
        shape, s = tuple(t.shape), t.stride()
        if len(shape) == 4:
            shape, s = (1, *shape), (0, *s)
        if len(shape) != 5 or shape[1] != n_pages:
            raise ValueError("pools must be [(L,) n_pages, Hkv, page_size, D]")
        _, _, h, r, d = shape
        if (d > 1 and s[4] != 1) or (r > 1 and s[3] != d) or (h > 1 and s[2] != r * d):
            raise ValueError("pools must have contiguous pages")
        _distinct_memory(t, "pools")
        size, page = t.element_size(), h * r * d
        arr += _POOL.pack(t.data_ptr(), (s[0] if shape[0] > 1 else 0) * size, (s[1] if n_pages > 1 else page) * size,
                          page * size, shape[0])
    return pools, arr


def paged_reserve(page_table: torch.Tensor, kv_lens: torch.Tensor, page_refs: torch.Tensor, n_new: torch.Tensor,
                  page_size: int, status: torch.Tensor | None = None,
                  guard: torch.Tensor | None = None) -> torch.Tensor:
    """Room for n_new (int32 [B], device) more tokens in every row of the table: the
    lowest free pages (page_refs 0) in the order of the rows; kv_lens grows by
    n_new. Behind a row that gets PAGED_NO_PAGES every row that needs a page gets it
    too, even if it needs fewer. Returns status int32 [B]: 0, PAGED_NO_PAGES or PAGED_TOO_LONG (that row
    unchanged: appended tokens would lie over the keys that it has, so it must bring
    none, or the append gets the guard of this call too). guard: int32 [4, B] on the
    device, zeros at first, then for paged_reserve and paged_append only."""
    B, W, row = _tables(page_table, kv_lens, page_refs)
    _ints(n_new, B, "n_new")
    if status is None:
        status = torch.empty(B, dtype=_I32, device=page_table.device)
    _ints(status, B, "status")
    used = [page_table, kv_lens, page_refs, n_new, status]
    held = _guard(guard, B, used)
    dev = _one_device("paged_reserve", *used)
    _call(lib.paged_reserve_guarded, "paged_reserve", dev, page_table.data_ptr(), row, kv_lens.data_ptr(),
          page_refs.data_ptr(), n_new.data_ptr(), status.data_ptr(), held, B, W, page_refs.numel(), int(page_size))
    return status


def paged_free(page_table: torch.Tensor, kv_lens: torch.Tensor, page_refs: torch.Tensor, rows) -> None:
    """The listed rows give up their pages (a page that no row holds any more is free) and become empty."""
    rows = _host_ints(rows, "rows")
    B, W, row = _tables(page_table, kv_lens, page_refs)
    dev = _one_device("paged_free", page_table, kv_lens, page_refs)
    _call(lib.paged_free, "paged_free", dev, page_table.data_ptr(), row, kv_lens.data_ptr(), page_refs.data_ptr(),
          rows.data_ptr(), rows.numel(), B, W, page_refs.numel())


def paged_fork(pools, page_table: torch.Tensor, kv_lens: torch.Tensor, page_refs: torch.Tensor, src, dst,
               status: torch.Tensor | None = None, page_size: int | None = None) -> torch.Tensor:
    """Empty rows dst become copies of rows src (src may repeat): whole pages shared,
    a partly filled last page copied in every pool (evicted pages stay evicted). Returns status int32 [n]: 0,
    PAGED_NO_PAGES or PAGED_IN_USE (that row unchanged)."""
    src, dst = _host_ints(src, "src"), _host_ints(dst, "dst")
    n = src.numel()
    _require(dst.numel() == n, "src and dst must have one length")
    B, W, row = _tables(page_table, kv_lens, page_refs)
    pools, arr = _pools(pools, page_refs.numel())
    if page_size is None:
        _require(len(pools) > 0 and len({t.shape[-2] for t in pools}) == 1, "pools of one page size, or page_size, needed")
        page_size = pools[0].shape[-2]
    if status is None:
        status = torch.empty(n, dtype=_I32, device=page_table.device)
    _ints(status, n, "status")
    dev = _one_device("paged_fork", page_table, kv_lens, page_refs, status, *pools)
    _call(lib.paged_fork, "paged_fork", dev, arr, len(pools), page_table.data_ptr(), row, kv_lens.data_ptr(),
          page_refs.data_ptr(), src.data_ptr(), dst.data_ptr(), status.data_ptr(), n, B, W, page_refs.numel(),
          int(page_size))
    return status


def paged_copy(pools, src, dst) -> None:
    """Page dst[i] becomes a copy of page src[i] in every pool (dst distinct, none in src)."""
    src, dst = _host_ints(src, "src"), _host_ints(dst, "dst")
    _require(src.numel() == dst.numel(), "src and dst must have one length")
    first = _slots(pools)[:1]
    _require(len(first) > 0 and first[0].dim() in (4, 5), "pools must be [(L,) n_pages, Hkv, page_size, D]")
    n_pages = first[0].shape[-4]
    pools, arr = _pools(pools, n_pages)
    dev = _one_device("paged_copy", *pools)
    _call(lib.paged_copy, "paged_copy", dev, arr, len(pools), src.data_ptr(), dst.data_ptr(), src.numel(), n_pages)


def paged_compact(pools, page_table: torch.Tensor, page_refs: torch.Tensor, out_table: torch.Tensor | None = None,
                  out_refs: torch.Tensor | None = None, n_live: torch.Tensor | None = None) -> torch.Tensor:
    """Moves the live pages to ids 0 .. n_live - 1 (the highest ids into the lowest
    free ones, both ascending); table and references follow, in place unless
    out_table / out_refs are given. Returns n_live, int32 [1] on the device."""
    B, W, row = _tables(page_table, None, page_refs)
    out_table = page_table if out_table is None else out_table
    out_refs = page_refs if out_refs is None else out_refs
    _require(_tables(out_table, None, out_refs) == (B, W, row) and out_refs.numel() == page_refs.numel(),
             "out_table and out_refs must be shaped like the inputs")
    if n_live is None:
        n_live = torch.empty(1, dtype=_I32, device=page_table.device)
    _ints(n_live, 1, "n_live")
    n_pages = page_refs.numel()
    pools, arr = _pools(pools, n_pages)
    need = lib.paged_compact_workspace_bytes(n_pages)
    _require(need > 0, "too many pages")
    workspace = torch.empty(need, dtype=torch.uint8, device=page_table.device)
    dev = _one_device("paged_compact", page_table, page_refs, out_table, out_refs, n_live, *pools)
    _call(lib.paged_compact, "paged_compact", dev, arr, len(pools), page_table.data_ptr(), out_table.data_ptr(), row,
          page_refs.data_ptr(), out_refs.data_ptr(), n_live.data_ptr(), workspace.data_ptr(), need, B, W, n_pages)
    return n_live


def paged_keep(pools, page_table: torch.Tensor, kv_lens: torch.Tensor, page_refs: torch.Tensor,
               cu_seqlens: torch.Tensor, path: torch.Tensor, n_keep: torch.Tensor, status: torch.Tensor | None = None,
               guard: torch.Tensor | None = None, page_size: int | None = None) -> torch.Tensor:
    """Of each row's last cu_seqlens[b + 1] - cu_seqlens[b] keys (a step's new tokens)
    only those listed in path[cu_seqlens[b] ..][:n_keep[b]] stay, strictly ascending numbers
    within them (draft_accept): moved together in every pool, kv_lens shortened,
    pages that are left empty given back. pools [(L,) n_pages,Hkv,page_size,D], and the
    scales of an 8-bit cache. Returns status int32 [B]: 0, or PAGED_BAD_PATH, PAGED_SHARED
    (a page that would be written, or that the row would end inside of, is another
    row's too) or PAGED_REFUSED (with a guard, that of the step: the row had no room for
    these tokens), that row unchanged."""
    B, W, row = _tables(page_table, kv_lens, page_refs)
    pools, arr = _pools(pools, page_refs.numel())
    if page_size is None:
        _require(len(pools) > 0 and len({t.shape[-2] for t in pools}) == 1, "pools of one page size, or page_size, needed")
        page_size = pools[0].shape[-2]
    _require(all(t.shape[-2] == page_size for t in pools), "the pools' pages must have page_size slots")
    heads = struct.pack(f"@{len(pools)}i", *[t.shape[-3] for t in pools])
    used, total = [page_table, kv_lens, page_refs, *pools], path.numel()
    at = _tokens(cu_seqlens, B + 1, "cu_seqlens", used), _tokens(path, total, "path", used), _tokens(n_keep, B, "n_keep", used)
    if status is None:
        status = torch.empty(B, dtype=_I32, device=page_table.device)
    to = _tokens(status, B, "status", used)
    held = _guard(guard, B, used)
    dev = _one_device("paged_keep", *used)
    _call(lib.paged_keep, "paged_keep", dev, arr, heads, len(pools), page_table.data_ptr(), row, kv_lens.data_ptr(),
          page_refs.data_ptr(), *at, to, held, total, B, W, page_refs.numel(), int(page_size))
    return status


class PagedCache:
    """A paged K/V cache of several layers that share one page table: pools bf16 (or,
    with dtype=torch.float8_e4m3fn, e4m3 with scales [layers, n_pages, Hkv, page_size])
    [layers, n_pages, Hkv, page_size, D], a table of `rows` sequences of up to
    max_pages pages, their lengths and the pages' reference counts.

    One serving step: reserve(n_new) once, then step(layer, ...) in every layer
    (append the new tokens, attend over the cache). fork / free / compact work on
    all layers at once. Rows without new tokens in a step have an empty range in
    cu_seqlens. A row that reserve refuses keeps its keys: the new tokens that a step
    brings for it all the same are dropped and see nothing (O = 0, lse = -inf).
    Everything runs on the current stream and can be captured (the row lists of fork
    and free are then part of the graph)."""

    def __init__(self, n_pages: int, Hkv: int, D: int, rows: int, max_pages: int, page_size: int = 16, layers: int = 1,
                 plan: RopePlan | None = None, interleaved: bool = False, device=None, dtype: torch.dtype = _BF16):
        _require(dtype in (_BF16, _E4M3), "a cache is bfloat16 or float8_e4m3fn")
        device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        shape = (layers, n_pages, Hkv, page_size, D)
        self.k_pages = torch.empty(shape, dtype=dtype, device=device)
        self.v_pages = torch.empty(shape, dtype=dtype, device=device)
        self.k_scales = self.v_scales = None
        if dtype == _E4M3:
            self.k_scales = torch.empty(shape[:-1], dtype=_E8M0, device=device)
            self.v_scales = torch.empty(shape[:-1], dtype=_E8M0, device=device)
        self.page_table = torch.full((rows, max_pages), -1, dtype=_I32, device=device)
        self.kv_lens = torch.zeros(rows, dtype=_I32, device=device)
        self.page_refs = torch.zeros(n_pages, dtype=_I32, device=device)
        self.guard = torch.zeros((4, rows), dtype=_I32, device=device)  # what reserve leaves for the steps
        self._step_lens = self.guard[3]
        self.page_size, self.plan, self.interleaved = page_size, plan, interleaved

    @property
    def _pools(self) -> tuple:
        pools = self.k_pages, self.v_pages
        return pools if self.k_scales is None else pools + (self.k_scales, self.v_scales)

    def reserve(self, n_new: torch.Tensor) -> torch.Tensor:
        return paged_reserve(self.page_table, self.kv_lens, self.page_refs, n_new, self.page_size, guard=self.guard)

    def step(self, layer: int, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
             positions: torch.Tensor | None = None, causal: bool = True, scale: float | None = None, workspace=None,
             tree: torch.Tensor | None = None):
        """Appends k, v [Hkv,total,D] (turned with q [Hq,total,D] by positions when
        the cache has a plan) and attends q over the cache: (O, lse). tree: the masks of
        new tokens that branch (draft_tree)."""
        pools = self.k_pages[layer], self.v_pages[layer]
        tables = self.page_table, self.kv_lens, cu_seqlens
        scales = {} if self.k_scales is None else {"k_scales": self.k_scales[layer], "v_scales": self.v_scales[layer]}
        if self.plan is None:
            _require(positions is None, "the cache has no plan to turn its keys by: positions are of no use to it")
            paged_append(k, v, *pools, *tables, guard=self.guard, **scales)
        else:
            _require(positions is not None, "the cache turns its keys by their positions: pass them")
            q = paged_append(k, v, *pools, *tables, q=q, positions=positions, inv_freq=self.plan.inv_freq,
                             axes=self.plan.axes, interleaved=self.interleaved, guard=self.guard, **scales)
        return attn_paged(q, *pools, self.page_table, self._step_lens, cu_seqlens, causal=causal, scale=scale,
                          workspace=workspace, tree=tree, **scales)

    def keep(self, cu_seqlens: torch.Tensor, path: torch.Tensor, n_keep: torch.Tensor) -> torch.Tensor:
        """Behind a step, in all layers: of its new tokens only those of the path stay (paged_keep)."""
        return paged_keep(self._pools, self.page_table, self.kv_lens, self.page_refs, cu_seqlens, path, n_keep,
                          guard=self.guard)

    def read(self, layer: int, cu_keys: torch.Tensor, total: int, first: torch.Tensor | None = None):
        """The keys and values of the rows, bf16 [Hkv,total,D] each (paged_read)."""
        scales = {} if self.k_scales is None else {"k_scales": self.k_scales[layer], "v_scales": self.v_scales[layer]}
        return paged_read(self.k_pages[layer], self.v_pages[layer], self.page_table, self.kv_lens, cu_keys, total, first,
                          **scales)

    def fork(self, src, dst) -> torch.Tensor:
        return paged_fork(self._pools, self.page_table, self.kv_lens, self.page_refs, src, dst)

    def free(self, rows) -> None:
        paged_free(self.page_table, self.kv_lens, self.page_refs, rows)

    def compact(self) -> torch.Tensor:
        return paged_compact(self._pools, self.page_table, self.page_refs)

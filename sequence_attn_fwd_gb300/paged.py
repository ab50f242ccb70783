"""The serving side: attention over a paged K/V cache, rotary positions with
several axes, appends to the cache and the management of its pages, over the C
ABI of include/seqattn_paged.h.

    plan = RopePlan(128, sections=(16, 24, 24))              # time, height, width
    q, k = rope_axes(q, k, positions, *plan)                 # training; gradients: rope_axes_bwd
    cache = PagedCache(n_pages=4096, Hkv=4, D=128, rows=64, max_pages=512, page_size=16, plan=plan)
    cache.reserve(n_new)                                      # room for the next tokens of every row
    o, lse = cache.step(0, q, k, v, cu_seqlens, positions)    # append, then attend (layer 0)
    cache.fork([0, 0], [8, 9]); cache.free([3]); cache.compact()

New tokens are packed: [H, total, D] tensors (any strides with D contiguous and
16-byte multiples, so a transposed [total, H, D] projection goes in without a
copy), sequence b in rows cu_seqlens[b] .. cu_seqlens[b + 1]. Page tables,
lengths, reference counts and cu_seqlens are int32 CUDA tensors, read on the
device: a captured call follows their contents. Lists of rows or pages are host
sequences (or CPU int32 tensors), checked before anything is launched.
"""
from __future__ import annotations

import contextlib
import ctypes
import math

import torch

from . import ATTN_BF16, ATTN_F32, _check, _require, _stream_handle
from ._lib import PagedCacheView, PagedPool, RopeRows, lib

PAGED_NO_PAGES, PAGED_TOO_LONG, PAGED_IN_USE = 1, 2, 3
_BF16, _I32 = torch.bfloat16, torch.int32


def _on(device: torch.device):
    """The device of the tensors as the current one (the kernels launch there)."""
    return contextlib.nullcontext() if torch.cuda.current_device() == device.index else torch.cuda.device(device)


def _one_device(what: str, *tensors):
    dev = tensors[0].device
    for t in tensors:
        _require(t.is_cuda and t.device == dev, f"{what}: all tensors must be on one CUDA device")
    return dev


def _host_ints(x, what: str) -> torch.Tensor:
    """A host list of ints as a contiguous int32 CPU tensor."""
    if not isinstance(x, torch.Tensor):
        x = torch.tensor([int(v) for v in x], dtype=_I32)
    _require(x.device.type == "cpu" and x.dtype == _I32 and x.dim() == 1, f"{what} must be host ints (or int32 CPU)")
    return x.contiguous()


def _ints(t: torch.Tensor, shape, what: str) -> None:
    _require(t.dtype == _I32 and tuple(t.shape) == tuple(shape) and t.is_contiguous(),
             f"{what} must be contiguous int32 {list(shape)}")


def _tables(page_table: torch.Tensor, kv_lens=None, page_refs=None) -> None:
    _require(page_table.dim() == 2 and page_table.dtype == _I32
             and (page_table.shape[1] <= 1 or page_table.stride(1) == 1), "page_table must be int32 [B, max_pages]")
    if kv_lens is not None:
        _ints(kv_lens, page_table.shape[:1], "kv_lens")
    if page_refs is not None:
        _require(page_refs.dtype == _I32 and page_refs.dim() == 1 and page_refs.is_contiguous() and page_refs.numel() > 0,
                 "page_refs must be contiguous int32 [n_pages]")


def _table_stride(t: torch.Tensor) -> int:
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _distinct_memory(t: torch.Tensor, what: str) -> None:
    """Every dimension longer than one has a non-zero stride (no expanded output)."""
    _require(all(n <= 1 or s != 0 for n, s in zip(t.shape, t.stride())), f"{what} must not be expanded")


def _packed(t: torch.Tensor, total: int, D: int, dtype, what: str) -> None:
    _require(t.dim() == 3 and t.shape[1] == total and t.shape[2] == D and t.dtype == dtype and t.is_cuda
             and t.stride(2) == 1, f"{what} must be {dtype} [H, {total}, {D}] with D contiguous")


def _cache_view(k_pages, v_pages, page_table, kv_lens, cu_seqlens) -> PagedCacheView:
    _require(k_pages.dim() == 4 and v_pages.shape == k_pages.shape, "pools must be [n_pages, Hkv, page_size, D]")
    n_pages, Hkv, ps, D = k_pages.shape
    for t in (k_pages, v_pages):
        _require(t.dtype == _BF16 and (n_pages == 0 or t[0].is_contiguous()), "pools must be bf16 with contiguous pages")
    stride = k_pages.stride(0) if n_pages > 1 else Hkv * ps * D
    _require(n_pages <= 1 or v_pages.stride(0) == stride, "the K and V pools must share their page stride")
    _tables(page_table, kv_lens)
    B = page_table.shape[0]
    _ints(cu_seqlens, (B + 1,), "cu_seqlens")
    _one_device("cache", k_pages, v_pages, page_table, kv_lens, cu_seqlens)
    return PagedCacheView(k_pages.data_ptr(), v_pages.data_ptr(), stride, page_table.data_ptr(),
                          _table_stride(page_table), kv_lens.data_ptr(), cu_seqlens.data_ptr(), B, n_pages, ps,
                          page_table.shape[1], Hkv, D)


def attn_paged_workspace_bytes(Hq: int, Hkv: int, total_q: int, D: int) -> int:
    """Device workspace bytes attn_paged needs."""
    n = lib.attn_paged_workspace_bytes(Hq, Hkv, total_q, D)
    _require(n > 0, "invalid sizes")
    return int(n)


def attn_paged(q: torch.Tensor, k_pages: torch.Tensor, v_pages: torch.Tensor, page_table: torch.Tensor,
               kv_lens: torch.Tensor, cu_seqlens: torch.Tensor, causal: bool = True, scale: float | None = None,
               out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
               workspace: torch.Tensor | None = None):
    """Attention of the packed new tokens q bf16 [Hq,total_q,D] over a paged cache.

    k_pages / v_pages bf16 [n_pages,Hkv,page_size,D]; page_table int32
    [B,max_pages] (an entry that is no page: its keys are not seen); kv_lens int32
    [B], the new tokens included (their keys are the last ones); cu_seqlens int32
    [B+1]. Under the causal mask token t of a sequence sees the keys up to its
    own. Returns (O bf16 [Hq,total_q,D], lse fp32 [Hq,total_q]); rows that see no
    key get O = 0, lse = -inf, rows of no sequence keep what out / lse held
    (unspecified where they are made here). workspace: a uint8 CUDA tensor of
    attn_paged_workspace_bytes(...), for one call at a time (made per call when
    not given)."""
    _require(q.dim() == 3, "expected q [Hq, total_q, D]")
    Hq, total, D = q.shape
    view = _cache_view(k_pages, v_pages, page_table, kv_lens, cu_seqlens)
    _require(view.D == D and Hq % view.Hkv == 0, "q must have the cache's D and a multiple of its heads")
    _packed(q, total, D, _BF16, "q")
    scale = 1.0 / math.sqrt(D) if scale is None else float(scale)
    if out is None:
        out = torch.empty((Hq, total, D), dtype=_BF16, device=q.device)
    if lse is None:
        lse = torch.empty((Hq, total), dtype=torch.float32, device=q.device)
    _packed(out, total, D, _BF16, "out")
    _distinct_memory(out, "out")
    _require(out.shape[0] == Hq, "bad out")
    _require(lse.shape == (Hq, total) and lse.dtype == torch.float32 and lse.is_contiguous(), "bad lse")
    if total == 0 or view.B == 0:
        return out, lse
    need = attn_paged_workspace_bytes(Hq, view.Hkv, total, D)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    _require(workspace.dtype == torch.uint8 and workspace.is_contiguous() and workspace.numel() >= need,
             "workspace must be a contiguous uint8 tensor of attn_paged_workspace_bytes(...) bytes")
    dev = _one_device("attn_paged", q, k_pages, out, lse, workspace)
    with _on(dev):
        st = lib.attn_paged(q.data_ptr(), q.stride(0), q.stride(1), ctypes.addressof(view), out.data_ptr(),
                            out.stride(0), out.stride(1), lse.data_ptr(), workspace.data_ptr(), workspace.numel(), Hq,
                            total, int(bool(causal)), scale, _stream_handle(dev))
    _check(st, "attn_paged")
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
    _require(inv_freq.device.type == "cpu" and inv_freq.dtype == torch.float64 and inv_freq.is_contiguous(),
             "inv_freq must be host floats (or float64 CPU)")
    _require(tuple(inv_freq.shape) == (D // 2,) and tuple(axes.shape) == (D // 2,), "inv_freq and axes need D / 2 entries")
    return inv_freq, axes


def _rope(q, k, positions, inv_freq, axes, interleaved, inverse, out_q, out_k):
    given = [t for t in (q, k) if t is not None]
    _require(len(given) > 0, "q or k is needed")
    B, _, S, D = given[0].shape
    dtype = given[0].dtype
    _require(dtype in (_BF16, torch.float32), "rows must be bf16 or fp32")
    views, outs = [], []
    for t, o in ((q, out_q), (k, out_k)):
        if t is None:
            views.append(None)
            outs.append(None)
            continue
        o = torch.empty(t.shape, dtype=dtype, device=t.device) if o is None else o
        for x in (t, o):
            _require(x.dim() == 4 and x.shape == t.shape and (x.shape[0], x.shape[2], x.shape[3]) == (B, S, D)
                     and x.dtype == dtype and x.is_cuda and x.stride(3) == 1,
                     "rows must be [B, H, S, D] of one dtype with D contiguous")
        _distinct_memory(o, "out")
        outs.append(o)
        views.append(RopeRows(t.data_ptr(), o.data_ptr(), t.stride(0), t.stride(1), t.stride(2), o.stride(0),
                              o.stride(1), o.stride(2), t.shape[1]))
    _require(positions.dim() == 3 and tuple(positions.shape[1:]) == (B, S) and positions.dtype == _I32
             and (S <= 1 or positions.stride(2) == 1), "positions must be int32 [n_axes, B, S]")
    inv_freq, axes = _plan(inv_freq, axes, D)
    dev = _one_device("rope_axes", positions, *given, *[o for o in outs if o is not None])
    with _on(dev):
        st = lib.rope_axes(*(None if v is None else ctypes.addressof(v) for v in views), positions.data_ptr(),
                           positions.stride(0), positions.stride(1), positions.shape[0], inv_freq.data_ptr(),
                           axes.data_ptr(), B, S, D, ATTN_F32 if dtype == torch.float32 else ATTN_BF16,
                           int(bool(interleaved)), int(inverse), _stream_handle(dev))
    _check(st, "rope_axes")
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
                 inv_freq=None, axes=None, interleaved: bool = False, out_q=None):
    """Writes the new tokens' k, v bf16 [Hkv,total,D] into the last slots of their
    sequences (kv_lens counts them already). With positions (int32
    [n_axes,total], inv_freq and axes as for rope_axes) k is turned on the way,
    and q [Hq,total,D] into out_q (may be q), which is returned. Tokens whose slot
    is on no page are dropped."""
    view = _cache_view(k_pages, v_pages, page_table, kv_lens, cu_seqlens)
    _require(k.dim() == 3, "expected k [Hkv, total, D]")
    total, D = k.shape[1], view.D
    _require(q is None or positions is not None, "q is turned by positions: pass them")
    rows = []
    for t, H in ((k, view.Hkv), (v, view.Hkv), (q, None)):
        if t is None:
            continue
        _packed(t, total, D, _BF16, "new tokens")
        _require(H is None or t.shape[0] == H, "k and v must have the cache's heads")
        rows.append(t)
    vq = None
    if q is not None:
        out_q = torch.empty(q.shape, dtype=_BF16, device=q.device) if out_q is None else out_q
        _packed(out_q, total, D, _BF16, "out_q")
        _require(out_q.shape == q.shape, "bad out_q")
        _distinct_memory(out_q, "out_q")
        rows.append(out_q)
        vq = RopeRows(q.data_ptr(), out_q.data_ptr(), 0, q.stride(0), q.stride(1), 0, out_q.stride(0), out_q.stride(1),
                      q.shape[0])
    vk = RopeRows(k.data_ptr(), None, 0, k.stride(0), k.stride(1), 0, 0, 0, view.Hkv)
    vv = RopeRows(v.data_ptr(), None, 0, v.stride(0), v.stride(1), 0, 0, 0, view.Hkv)
    pos, pos_axis, n_axes, f, a = None, 0, 0, None, None
    if positions is not None:
        _require(positions.dim() == 2 and positions.shape[1] == total and positions.dtype == _I32
                 and (total <= 1 or positions.stride(1) == 1), "positions must be int32 [n_axes, total]")
        inv_freq, axes = _plan(inv_freq, axes, D)
        pos, pos_axis, n_axes, f, a = (positions.data_ptr(), positions.stride(0), positions.shape[0],
                                       inv_freq.data_ptr(), axes.data_ptr())
        rows.append(positions)
    dev = _one_device("paged_append", k_pages, *rows)
    with _on(dev):
        st = lib.paged_append(None if vq is None else ctypes.addressof(vq), ctypes.addressof(vk), ctypes.addressof(vv),
                              ctypes.addressof(view), pos, pos_axis, n_axes, f, a, total, int(bool(interleaved)),
                              _stream_handle(dev))
    _check(st, "paged_append")
    return out_q


def _pools(pools, n_pages: int):
    """Pools [n_pages,Hkv,page_size,D] or [L,n_pages,Hkv,page_size,D] (one tensor or several) as paged_pool."""
    pools = (pools,) if isinstance(pools, torch.Tensor) else tuple(pools)
    arr = (PagedPool * max(len(pools), 1))()
    for i, t in enumerate(pools):
        _require(t.dim() in (4, 5) and t.shape[-4] == n_pages, "pools must be [(L,) n_pages, Hkv, page_size, D]")
        layers = t if t.dim() == 5 else t[None]
        _require(layers.numel() == 0 or layers[0, 0].is_contiguous(), "pages must be contiguous")
        _distinct_memory(t, "pools")
        size = t.element_size()
        page = layers.shape[2] * layers.shape[3] * layers.shape[4]
        arr[i] = PagedPool(t.data_ptr(), (layers.stride(0) if layers.shape[0] > 1 else 0) * size,
                           (layers.stride(1) if n_pages > 1 else page) * size, page * size, layers.shape[0])
    return pools, arr


def paged_reserve(page_table: torch.Tensor, kv_lens: torch.Tensor, page_refs: torch.Tensor, n_new: torch.Tensor,
                  page_size: int, status: torch.Tensor | None = None) -> torch.Tensor:
    """Room for n_new (int32 [B], device) more tokens in every row of the table: the
    lowest free pages (page_refs 0) in the order of the rows; kv_lens grows by
    n_new. Returns status int32 [B]: 0, PAGED_NO_PAGES or PAGED_TOO_LONG (that row
    unchanged)."""
    _tables(page_table, kv_lens, page_refs)
    B, W = page_table.shape
    _ints(n_new, (B,), "n_new")
    status = torch.empty(B, dtype=_I32, device=page_table.device) if status is None else status
    _ints(status, (B,), "status")
    dev = _one_device("paged_reserve", page_table, kv_lens, page_refs, n_new, status)
    with _on(dev):
        st = lib.paged_reserve(page_table.data_ptr(), _table_stride(page_table), kv_lens.data_ptr(), page_refs.data_ptr(),
                               n_new.data_ptr(), status.data_ptr(), B, W, page_refs.numel(), int(page_size),
                               _stream_handle(dev))
    _check(st, "paged_reserve")
    return status


def paged_free(page_table: torch.Tensor, kv_lens: torch.Tensor, page_refs: torch.Tensor, rows) -> None:
    """The listed rows give up their pages (a page that no row holds any more is free) and become empty."""
    rows = _host_ints(rows, "rows")
    _tables(page_table, kv_lens, page_refs)
    B, W = page_table.shape
    dev = _one_device("paged_free", page_table, kv_lens, page_refs)
    with _on(dev):
        st = lib.paged_free(page_table.data_ptr(), _table_stride(page_table), kv_lens.data_ptr(), page_refs.data_ptr(),
                            rows.data_ptr(), rows.numel(), B, W, page_refs.numel(), _stream_handle(dev))
    _check(st, "paged_free")


def paged_fork(pools, page_table: torch.Tensor, kv_lens: torch.Tensor, page_refs: torch.Tensor, src, dst,
               status: torch.Tensor | None = None, page_size: int | None = None) -> torch.Tensor:
    """Empty rows dst become copies of rows src (src may repeat): whole pages shared,
    a partly filled last page copied in every pool. Returns status int32 [n]: 0,
    PAGED_NO_PAGES or PAGED_IN_USE (that row unchanged)."""
    src, dst = _host_ints(src, "src"), _host_ints(dst, "dst")
    _require(src.numel() == dst.numel(), "src and dst must have one length")
    _tables(page_table, kv_lens, page_refs)
    B, W = page_table.shape
    pools, arr = _pools(pools, page_refs.numel())
    if page_size is None:
        _require(len(pools) > 0 and len({t.shape[-2] for t in pools}) == 1, "pools of one page size, or page_size, needed")
        page_size = pools[0].shape[-2]
    status = torch.empty(src.numel(), dtype=_I32, device=page_table.device) if status is None else status
    _ints(status, (src.numel(),), "status")
    dev = _one_device("paged_fork", page_table, kv_lens, page_refs, status, *pools)
    with _on(dev):
        st = lib.paged_fork(ctypes.addressof(arr), len(pools), page_table.data_ptr(), _table_stride(page_table),
                            kv_lens.data_ptr(), page_refs.data_ptr(), src.data_ptr(), dst.data_ptr(), status.data_ptr(),
                            src.numel(), B, W, page_refs.numel(), int(page_size), _stream_handle(dev))
    _check(st, "paged_fork")
    return status


def paged_copy(pools, src, dst) -> None:
    """Page dst[i] becomes a copy of page src[i] in every pool (dst distinct, none in src)."""
    src, dst = _host_ints(src, "src"), _host_ints(dst, "dst")
    _require(src.numel() == dst.numel(), "src and dst must have one length")
    first = pools if isinstance(pools, torch.Tensor) else pools[0]
    n_pages = first.shape[-4]
    pools, arr = _pools(pools, n_pages)
    dev = _one_device("paged_copy", *pools)
    with _on(dev):
        st = lib.paged_copy(ctypes.addressof(arr), len(pools), src.data_ptr(), dst.data_ptr(), src.numel(), n_pages,
                            _stream_handle(dev))
    _check(st, "paged_copy")


def paged_compact(pools, page_table: torch.Tensor, page_refs: torch.Tensor, out_table: torch.Tensor | None = None,
                  out_refs: torch.Tensor | None = None, n_live: torch.Tensor | None = None) -> torch.Tensor:
    """Moves the live pages to ids 0 .. n_live - 1 (the highest ids into the lowest
    free ones, both ascending); table and references follow, in place unless
    out_table / out_refs are given. Returns n_live, int32 [1] on the device."""
    _tables(page_table, None, page_refs)
    B, W = page_table.shape
    out_table = page_table if out_table is None else out_table
    out_refs = page_refs if out_refs is None else out_refs
    _tables(out_table, None, out_refs)
    _require(out_table.shape == page_table.shape and _table_stride(out_table) == _table_stride(page_table)
             and out_refs.shape == page_refs.shape, "out_table and out_refs must be shaped like the inputs")
    n_live = torch.empty(1, dtype=_I32, device=page_table.device) if n_live is None else n_live
    _ints(n_live, (1,), "n_live")
    n_pages = page_refs.numel()
    pools, arr = _pools(pools, n_pages)
    need = lib.paged_compact_workspace_bytes(n_pages)
    _require(need > 0, "too many pages")
    workspace = torch.empty(need, dtype=torch.uint8, device=page_table.device)
    dev = _one_device("paged_compact", page_table, page_refs, out_table, out_refs, n_live, *pools)
    with _on(dev):
        st = lib.paged_compact(ctypes.addressof(arr), len(pools), page_table.data_ptr(), out_table.data_ptr(),
                               _table_stride(page_table), page_refs.data_ptr(), out_refs.data_ptr(), n_live.data_ptr(),
                               workspace.data_ptr(), need, B, W, n_pages, _stream_handle(dev))
    _check(st, "paged_compact")
    return n_live


class PagedCache:
    """A paged K/V cache of several layers that share one page table: pools bf16
    [layers, n_pages, Hkv, page_size, D], a table of `rows` sequences of up to
    max_pages pages, their lengths and the pages' reference counts.

    One serving step: reserve(n_new) once, then step(layer, ...) in every layer
    (append the new tokens, attend over the cache). fork / free / compact work on
    all layers at once. Rows without new tokens in a step have an empty range in
    cu_seqlens. Everything runs on the current stream and can be captured (the
    row lists of fork and free are then part of the graph)."""

    def __init__(self, n_pages: int, Hkv: int, D: int, rows: int, max_pages: int, page_size: int = 16, layers: int = 1,
                 plan: RopePlan | None = None, interleaved: bool = False, device=None):
        device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
        shape = (layers, n_pages, Hkv, page_size, D)
        self.k_pages = torch.empty(shape, dtype=_BF16, device=device)
        self.v_pages = torch.empty(shape, dtype=_BF16, device=device)
        self.page_table = torch.full((rows, max_pages), -1, dtype=_I32, device=device)
        self.kv_lens = torch.zeros(rows, dtype=_I32, device=device)
        self.page_refs = torch.zeros(n_pages, dtype=_I32, device=device)
        self.page_size, self.plan, self.interleaved = page_size, plan, interleaved

    def reserve(self, n_new: torch.Tensor) -> torch.Tensor:
        return paged_reserve(self.page_table, self.kv_lens, self.page_refs, n_new, self.page_size)

    def step(self, layer: int, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
             positions: torch.Tensor | None = None, causal: bool = True, scale: float | None = None, workspace=None):
        """Appends k, v [Hkv,total,D] (turned with q [Hq,total,D] by positions when
        the cache has a plan) and attends q over the cache: (O, lse)."""
        pools = self.k_pages[layer], self.v_pages[layer]
        tables = self.page_table, self.kv_lens, cu_seqlens
        if self.plan is None:
            paged_append(k, v, *pools, *tables)
        else:
            _require(positions is not None, "the cache turns its keys by their positions: pass them")
            q = paged_append(k, v, *pools, *tables, q=q, positions=positions, inv_freq=self.plan.inv_freq,
                             axes=self.plan.axes, interleaved=self.interleaved)
        return attn_paged(q, *pools, *tables, causal=causal, scale=scale, workspace=workspace)

    def fork(self, src, dst) -> torch.Tensor:
        return paged_fork((self.k_pages, self.v_pages), self.page_table, self.kv_lens, self.page_refs, src, dst)

    def free(self, rows) -> None:
        paged_free(self.page_table, self.kv_lens, self.page_refs, rows)

    def compact(self) -> torch.Tensor:
        return paged_compact((self.k_pages, self.v_pages), self.page_table, self.page_refs)

"""The serving-side entry points of include/seqattn_paged.h: exported, declared, and refusing bad arguments on the
host, before any CUDA call (no GPU needed)."""
import ctypes
import os
import re

import pytest
import torch

from tests.test_abi import FAKE, ROOT, build_mod

HEADER = os.path.join(ROOT, "include", "seqattn_paged.h")
F = ctypes.c_float


@pytest.fixture(scope="module")
def lib():
    path = build_mod.build()
    from sequence_attn_fwd_gb300._lib import load

    return load(path)


def test_declared_functions_are_exported(lib):
    from sequence_attn_fwd_gb300._lib import PAGED_EXPORTS

    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    declared = sorted(set(re.findall(r"^\s*(?:int|size_t)\s+(\w+)\s*\(", text, flags=re.M)))
    assert declared == sorted(PAGED_EXPORTS)
    for name in declared:
        assert hasattr(lib, name), name


def test_struct_sizes_match_the_header(lib):
    from sequence_attn_fwd_gb300._lib import PagedCacheView, PagedPool, RopeRows

    assert ctypes.sizeof(PagedCacheView) == 7 * 8 + 6 * 4
    assert ctypes.sizeof(RopeRows) == 8 * 8 + 8
    assert ctypes.sizeof(PagedPool) == 4 * 8 + 8


def view(**kw):
    from sequence_attn_fwd_gb300._lib import PagedCacheView

    d = dict(k_pages=FAKE, v_pages=FAKE, page_stride=2 * 16 * 128, page_table=FAKE, table_stride=8, kv_lens=FAKE,
             cu_seqlens=FAKE, B=2, n_pages=8, page_size=16, max_pages=8, Hkv=2, D=128)
    d.update(kw)
    return PagedCacheView(**d)


def test_attn_paged_refusals(lib):
    ws = lib.attn_paged_workspace_bytes(4, 2, 5, 128)
    assert ws > 0

    def run(q=FAKE, qh=5 * 128, qr=128, o=FAKE, lse=FAKE, w=FAKE, wb=ws, Hq=4, total=5, causal=1, scale=0.1, **kw):
        v = view(**kw)
        return lib.attn_paged(q, qh, qr, ctypes.addressof(v), o, qh, qr, lse, w, wb, Hq, total, causal, F(scale), None)

    assert run(D=96) == 2 and run(D=256) == 2
    assert run(page_size=8) == 2 and run(page_size=24) == 2 and run(page_size=0) == 1
    assert run(max_pages=1 << 27, table_stride=1 << 27) == 2  # more than 2^30 keys
    assert run(total=1 << 29, wb=1 << 40, B=4096, max_pages=1 << 26, table_stride=1 << 26) == 2  # key tiles past 2^31
    assert run(B=4097) == 2 and run(Hq=512) == 2  # too many sequences; more than 128 heads in a group
    assert run(Hq=3) == 1 and run(causal=2) == 1 and run(scale=0.0) == 1 and run(scale=float("inf")) == 1
    assert run(page_stride=16 * 128) == 1 and run(page_stride=2 * 16 * 128 + 4) == 1 and run(table_stride=7) == 1
    assert run(q=0) == 1 and run(q=FAKE + 8) == 1 and run(o=FAKE + 2) == 1 and run(lse=FAKE + 2) == 1
    assert run(qr=129) == 1 and run(qr=64) == 1 and run(qh=0) == 1
    assert run(w=0) == 1 and run(w=FAKE + 8) == 1 and run(wb=ws - 1) == 1
    assert run(k_pages=0) == 1 and run(v_pages=FAKE + 8) == 1 and run(page_table=0) == 1 and run(cu_seqlens=FAKE + 1) == 1
    assert run(n_pages=0) == 1 and run(Hkv=0) == 1 and run(total=-1) == 1
    assert run(total=0) == 0 and run(B=0) == 0
    assert lib.attn_paged(FAKE, 640, 128, None, FAKE, 640, 128, None, FAKE, ws, 4, 5, 1, F(0.1), None) == 1


def test_attn_paged_workspace(lib):
    up = lambda n: (n + 255) // 256 * 256
    want = lambda rows, D: up(320 * rows * D * 4) + up(320 * rows * 4) + up(160 * 16)
    assert lib.attn_paged_workspace_bytes(28, 4, 1, 128) == want(7, 128)       # one token: a group's rows
    assert lib.attn_paged_workspace_bytes(28, 4, 10 ** 6, 128) == want(252, 128)  # two tiles of 18 tokens
    assert lib.attn_paged_workspace_bytes(8, 8, 10 ** 6, 64) == want(256, 64)
    for bad in ((3, 2, 1, 128), (4, 2, 1, 96), (0, 1, 1, 64), (256, 1, 1, 64), (4, 2, -1, 64)):
        assert lib.attn_paged_workspace_bytes(*bad) == 0


def rope_args(D=128, freq=None, axes=None):
    f = (ctypes.c_double * (D // 2))(*(freq or [0.5] * (D // 2)))
    a = (ctypes.c_int * (D // 2))(*(axes or [0] * (D // 2)))
    return f, a


def rows(heads=2, at=FAKE, out=FAKE, s=128):
    from sequence_attn_fwd_gb300._lib import RopeRows

    return RopeRows(at, out, 64 * 128 * heads, 64 * 128, s, 64 * 128 * heads, 64 * 128, s, heads)


def test_rope_axes_refusals(lib):
    def run(q=None, pos=FAKE, n_axes=3, B=2, S=64, D=128, dtype=0, inter=0, inv=0, freq=None, axes=None):
        q = rows() if q is None else q
        f, a = rope_args(128, freq, axes)
        return lib.rope_axes(ctypes.addressof(q), None, pos, 128, 64, n_axes, ctypes.addressof(f), ctypes.addressof(a), B,
                             S, D, dtype, inter, inv, None)

    assert run(D=96) == 2 and run(dtype=2) == 1 and run(inter=2) == 1 and run(inv=-1) == 1
    assert run(axes=[3] + [0] * 63) == 1 and run(axes=[-2] + [0] * 63) == 1 and run(n_axes=0) == 1
    assert run(freq=[float("nan")] + [0.1] * 63) == 1 and run(freq=[float("inf")] + [0.1] * 63) == 1
    assert run(pos=0) == 1 and run(pos=FAKE + 2) == 1 and run(B=-1) == 1
    assert run(q=rows(at=FAKE + 8)) == 1 and run(q=rows(out=0)) == 1 and run(q=rows(s=132)) == 1 and run(q=rows(heads=-1)) == 1
    assert run(B=1 << 16, S=1 << 16) == 2
    assert run(B=0) == 0 and run(S=0) == 0
    assert run(q=rows(heads=0)) == 0  # nothing to turn


def test_paged_append_refusals(lib):
    def run(k=None, v=None, q=None, pos=FAKE, total=9, inter=0, axes=None, **kw):
        c = view(**kw)
        k, v = rows() if k is None else k, rows() if v is None else v
        f, a = rope_args(128, None, axes)
        return lib.paged_append(None if q is None else ctypes.addressof(q), ctypes.addressof(k), ctypes.addressof(v),
                                ctypes.addressof(c), pos, 64, 3, ctypes.addressof(f), ctypes.addressof(a), total, inter, None)

    assert run(D=80) == 2 and run(page_size=12) == 2 and run(B=4097) == 2
    assert run(k=rows(heads=3)) == 1 and run(v=rows(heads=1)) == 1 and run(total=-1) == 1 and run(inter=3) == 1
    assert run(q=rows(4), pos=0) == 1  # q without positions
    assert run(q=rows(4, out=FAKE + 4)) == 1 and run(k=rows(at=FAKE + 2)) == 1 and run(pos=FAKE + 1) == 1
    assert run(axes=[5] * 64) == 1
    assert run(total=0) == 0 and run(B=0) == 0


def ints(*x):
    return (ctypes.c_int * max(1, len(x)))(*x)


def pool(n=1, **kw):
    from sequence_attn_fwd_gb300._lib import PagedPool

    d = dict(base=FAKE, layer_stride=1 << 16, page_stride=4096, page_bytes=4096, n_layers=2)
    d.update(kw)
    return (PagedPool * n)(*[PagedPool(**d) for _ in range(n)])


def test_page_management_refusals(lib):
    A = ctypes.addressof

    def reserve(table=FAKE, stride=8, lens=FAKE, status=FAKE, B=4, W=8, n=16, ps=16):
        return lib.paged_reserve(table, stride, lens, FAKE, FAKE, status, B, W, n, ps, None)

    assert reserve(ps=8) == 2 and reserve(ps=48) == 2 and reserve(ps=-16) == 1 and reserve(B=4097) == 2
    assert reserve(stride=7) == 1 and reserve(table=0) == 1 and reserve(lens=FAKE + 2) == 1 and reserve(status=0) == 1
    assert reserve(n=0) == 1 and reserve(W=1 << 27, stride=1 << 27) == 2 and reserve(B=0) == 0

    def free(*r, B=4):
        x = ints(*r)
        return lib.paged_free(FAKE, 8, FAKE, FAKE, A(x), len(r), B, 8, 16, None)

    assert free(4) == 1 and free(-1) == 1 and free(1, 2, 1) == 1 and free() == 0
    assert lib.paged_free(FAKE, 8, FAKE, FAKE, None, 1, 4, 8, 16, None) == 1

    def fork(src, dst, pools=None, n_pools=1, ps=16, status=FAKE):
        pools = pool() if pools is None else pools
        s, d = ints(*src), ints(*dst)
        return lib.paged_fork(A(pools), n_pools, FAKE, 8, FAKE, FAKE, A(s), A(d), status, len(src), 8, 8, 16, ps, None)

    assert fork([0, 0], [1, 1]) == 1  # one target twice
    assert fork([0, 1], [1, 2]) == 1  # a target that is also a source
    assert fork([0], [8]) == 1 and fork([-1], [1]) == 1 and fork([0], [1], ps=10) == 2 and fork([0], [1], status=0) == 1
    assert fork([0], [1], pool(base=FAKE + 8)) == 1 and fork([0], [1], pool(page_bytes=24)) == 1
    assert fork([0], [1], pool(page_stride=2048)) == 1 and fork([0], [1], pool(n_layers=-1)) == 1
    assert fork([0], [1], pool(33), 33) == 2 and fork([], []) == 0

    def copy(src, dst, n_pages=100000, pools=None):
        pools = pool() if pools is None else pools
        s, d = ints(*src), ints(*dst)
        return lib.paged_copy(A(pools), 1, A(s), A(d), len(src), n_pages, None)

    assert copy([0, 1], [2, 2]) == 1 and copy([0, 1], [1, 2]) == 1 and copy([0], [0]) == 1
    assert copy([0, 99999], [99998, 99999]) == 1  # far apart
    assert copy([100000], [1]) == 1 and copy([1], [-1]) == 1 and copy([], []) == 0
    assert copy([0], [1], pools=pool(n_layers=0)) == 0  # nothing to copy

    need = lib.paged_compact_workspace_bytes(16)
    assert need > 0 and lib.paged_compact_workspace_bytes(0) == 0 and lib.paged_compact_workspace_bytes(-4) == 0

    def compact(out=FAKE, n_live=FAKE, ws=FAKE, wb=need, n=16, refs=FAKE):
        pools = pool()
        return lib.paged_compact(A(pools), 1, FAKE, out, 8, refs, FAKE, n_live, ws, wb, 4, 8, n, None)

    assert compact(out=0) == 1 and compact(n_live=0) == 1 and compact(ws=0) == 1 and compact(wb=need - 1) == 1
    assert compact(n=0) == 1 and compact(refs=FAKE + 2) == 1


def test_wrappers_refuse_bad_tensors():
    """Shape, type and layout checks come before anything touches a GPU."""
    import sequence_attn_fwd_gb300 as sa

    bf, i32 = torch.bfloat16, torch.int32
    q = torch.zeros((4, 5, 128), dtype=bf)
    kp = torch.zeros((8, 2, 16, 128), dtype=bf)
    table, lens, cu = torch.zeros((2, 4), dtype=i32), torch.zeros(2, dtype=i32), torch.zeros(3, dtype=i32)
    with pytest.raises(ValueError, match="cu_seqlens"):
        sa.attn_paged(q, kp, kp, table, lens, torch.zeros(2, dtype=i32))
    with pytest.raises(ValueError, match="pools"):
        sa.attn_paged(q, kp, kp[:, :1], table, lens, cu)
    with pytest.raises(ValueError, match="pools"):
        sa.attn_paged(q, kp.transpose(1, 2), kp.transpose(1, 2), table, lens, cu)
    with pytest.raises(ValueError, match="page_table"):
        sa.attn_paged(q, kp, kp, table.long(), lens, cu)
    with pytest.raises(ValueError, match="CUDA"):
        sa.attn_paged(q, kp, kp, table, lens, cu)  # right shapes, but not on a GPU
    with pytest.raises(ValueError, match="sections"):
        sa.RopePlan(64, (16, 24))
    with pytest.raises(ValueError, match="rows must be"):
        sa.rope_axes(q[None].half(), None, torch.zeros((1, 1, 5), dtype=i32), *sa.RopePlan(128))
    with pytest.raises(ValueError, match="host ints"):
        sa.paged_free(table, lens, torch.zeros(8, dtype=i32), torch.zeros(1))
    with pytest.raises(ValueError, match="one length"):
        sa.paged_copy(kp, [1, 2], [3])


def test_rope_plan_frequencies():
    import sequence_attn_fwd_gb300 as sa

    f, a = sa.RopePlan(128, (16, 24, 20), base=5000.0)
    assert a.tolist() == [0] * 16 + [1] * 24 + [2] * 20 + [-1] * 4
    assert f[17].item() == pytest.approx(5000.0 ** (-34 / 128)) and f[63].item() == 0.0
    f, a = sa.RopePlan(64, (16, 16), shared=False)
    assert f[0].item() == f[16].item() == 1.0 and f[20].item() == pytest.approx(10000.0 ** (-4 / 16))


def test_host_model_of_the_tables():
    """The model that the GPU tests compare with, on cases small enough to check by hand."""
    from tests.paged_ref import Tables

    t = Tables([[-1] * 4 for _ in range(4)], [0, 0, 0, 0], [0] * 6, 16)
    assert t.reserve([33, 16, 0, 0]) == [0, 0, 0, 0] and t.table[0][:3] == [0, 1, 2] and t.table[1][0] == 3
    assert t.fork([0, 0], [2, 3]) == ([0, 0], [(2, 4), (2, 5)]) and t.refs == [3, 3, 1, 1, 1, 1]
    assert t.reserve([15, 1, 0, 40]) == [0, 1, 0, 2] and t.lens == [48, 16, 33, 33]
    t.free([0, 3])
    assert t.refs == [1, 1, 0, 1, 1, 0]
    assert t.compact() == (4, [(4, 2)]) and t.table[2] == [0, 1, 2, -1] and t.refs == [1, 1, 1, 1, 0, 0]

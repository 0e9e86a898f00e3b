"""Host-side refusals of the entry points on pages: bad arguments are turned
down before anything reaches the GPU (no launch here)."""

import ctypes
import os

import pytest
import torch

from wavelet_guided_sparse_gb300 import binding as bd

OK, NULL, SHAPE, UNSUPPORTED, WORKSPACE, ALIGNMENT = 0, 1, 2, 3, 4, 7
P = ctypes.c_void_p(1 << 20)          # aligned, never dereferenced
ODD2 = ctypes.c_void_p((1 << 20) + 2)
ODD4 = ctypes.c_void_p((1 << 20) + 4)
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(bd.LIB_PATH):
        from wavelet_guided_sparse_gb300 import build
        build.build()
    return bd.lib()


def dims(**kw):
    base = dict(n_seqs=4, q_heads=1, kv_heads=2, head_dim=128, page_size=16, n_pages=100,
                table_pages=20, dtype=0)
    base.update(kw)
    return ctypes.byref(bd.PageDims(**base))


def pools(*at):
    return (ctypes.c_void_p * max(len(at), 1))(*at), len(at)


def reserve(lib, d=None, rows=P, refs=P, table=P, ws=P, wsb=BIG):
    return lib.wf_paged_reserve(d or dims(), rows, refs, table, ws, wsb, None)


def fork(lib, d=None, n=2, src=P, dst=P, lens=P, share=None, refs=P, table=P, p=(P, P), ws=P,
         wsb=BIG, count=None):
    at, k = pools(*[x.value if x is not None else None for x in p])
    return lib.wf_paged_fork(d or dims(), n, src, dst, lens, share, refs, table,
                             k if count is None else count, at, ws, wsb, None)


def keep(lib, d=None, lens=P, start=P, rows=P, most=3, n=P, refs=P, table=P, p=(P, P), ws=P,
         wsb=BIG):
    at, k = pools(*[x.value if x is not None else None for x in p])
    return lib.wf_paged_keep(d or dims(), lens, start, rows, most, n, refs, table, k, at, ws, wsb,
                             None)


def release(lib, d=None, first=P, end=P, refs=P, table=P, ws=None, wsb=0):
    return lib.wf_paged_release(d or dims(), first, end, refs, table, ws, wsb, None)


BAD = [(dict(head_dim=96), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED), (dict(kv_heads=0), SHAPE),
       (dict(n_seqs=0), SHAPE), (dict(n_seqs=4097), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED),
       (dict(n_pages=1 << 27), UNSUPPORTED), (dict(table_pages=0), SHAPE)]


@pytest.mark.parametrize("kw,want", BAD)
def test_sizes(lib, kw, want):
    n = ctypes.c_size_t(0)
    assert lib.wf_pages_workspace_bytes(dims(**kw), 0, 0, ctypes.byref(n)) == want
    for call in (reserve, fork, keep, release):
        assert call(lib, dims(**kw)) == want


def test_query_heads_are_not_looked_at(lib):
    n = ctypes.c_size_t(0)
    for q in (0, -1, 7, 1 << 20):
        assert lib.wf_pages_workspace_bytes(dims(q_heads=q), 0, 0, ctypes.byref(n)) == OK


def test_workspace(lib):
    n = ctypes.c_size_t(0)
    got = []
    for forks, rows in ((0, 0), (3, 0), (0, 5), (4096, 320), (0, 320)):
        assert lib.wf_pages_workspace_bytes(dims(), forks, rows, ctypes.byref(n)) == OK
        got.append(n.value)
    assert 256 < got[0] < got[1] < got[3] and got[0] < got[4]
    assert lib.wf_pages_workspace_bytes(dims(), -1, 0, ctypes.byref(n)) == SHAPE
    assert lib.wf_pages_workspace_bytes(dims(), 4097, 0, ctypes.byref(n)) == UNSUPPORTED
    assert lib.wf_pages_workspace_bytes(dims(), 0, 321, ctypes.byref(n)) == SHAPE
    assert lib.wf_pages_workspace_bytes(dims(), 0, -1, ctypes.byref(n)) == SHAPE
    assert lib.wf_pages_workspace_bytes(dims(), 0, 0, None) == NULL
    assert lib.wf_pages_workspace_bytes(None, 0, 0, ctypes.byref(n)) == NULL
    assert reserve(lib, wsb=got[0] - 1) == WORKSPACE
    assert fork(lib, wsb=got[0]) == WORKSPACE
    assert keep(lib, wsb=256) == WORKSPACE
    assert release(lib, ws=P, wsb=255) == WORKSPACE


def test_pointers(lib):
    for call, names in ((reserve, ("rows", "refs", "table", "ws")),
                        (fork, ("src", "dst", "lens", "refs", "table", "ws")),
                        (keep, ("lens", "start", "table", "ws", "rows", "n")),
                        (release, ("first", "end", "refs", "table"))):
        for name in names:
            assert call(lib, **{name: None}) == NULL, (call, name)
            if name != "ws":
                assert call(lib, **{name: ODD2}) == ALIGNMENT, (call, name)
        if call is not release:
            assert call(lib, ws=ODD4) == ALIGNMENT
    assert fork(lib, share=ODD2) == ALIGNMENT
    assert keep(lib, refs=ODD2) == ALIGNMENT
    assert release(lib, ws=ODD4, wsb=BIG) == ALIGNMENT
    assert keep(lib, rows=None, n=None, refs=None) == NULL     # nothing to move, nothing to free


def test_pools_and_counts(lib):
    for call in (fork, keep):
        assert call(lib, p=()) == SHAPE
        assert call(lib, p=(P,) * 257) == UNSUPPORTED
        assert call(lib, p=(P, None)) == NULL
        assert call(lib, p=(P, ODD4)) == ALIGNMENT
    assert fork(lib, n=-1) == SHAPE
    assert fork(lib, n=4097) == UNSUPPORTED
    assert fork(lib, n=0, src=None, dst=None) == OK            # nothing launched
    assert keep(lib, most=-1) == SHAPE
    assert keep(lib, most=321) == SHAPE


def test_binding_refuses_cpu_tensors():
    x = torch.zeros((4, 2, 16, 64))
    cache, i = {"K": x, "V": x}, torch.zeros(3, dtype=torch.int32)
    table = torch.full((3, 5), -1, dtype=torch.int32)
    for call in (lambda: bd.paged_reserve(cache, table, i, i),
                 lambda: bd.paged_fork(cache, table, i, i, i, i),
                 lambda: bd.paged_keep(cache, table, i, i),
                 lambda: bd.paged_release(cache, table, i, i, i),
                 lambda: bd.page_pools(cache), lambda: bd.page_pools([]),
                 lambda: bd.alloc_pages_workspace(cache, table)):
        with pytest.raises(ValueError):
            call()

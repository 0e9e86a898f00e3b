"""Host-side refusals of the windowed and the tree attention (no launch here)."""

import ctypes
import os

import pytest
import torch

from test_abi_dense import BAD_DIMS, NULL, ALIGNMENT, ODD, ODD2, OK, P, SHAPE, UNSUPPORTED, WORKSPACE
from test_abi_dense import opts, pages
from wavelet_guided_sparse_gb300 import binding as bd


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(bd.LIB_PATH):
        from wavelet_guided_sparse_gb300 import build
        build.build()
    return bd.lib()


def window(lib, dims, o, window=10, sinks=0, new=1, q=P, k=P, v=P, table=P, lens=P, out=P,
           lse=None, ws=P, wsb=1 << 40):
    return lib.wf_paged_window_attn(ctypes.byref(dims), ctypes.byref(o) if o is not None else None,
                                    window, sinks, new, q, k, v, table, lens, out, lse, ws, wsb,
                                    None)


def tree(lib, dims, o, new=1, q=P, k=P, v=P, table=P, lens=P, parents=P, count=None, out=P,
         lse=None, ws=P, wsb=1 << 40):
    return lib.wf_paged_tree_attn(ctypes.byref(dims), ctypes.byref(o) if o is not None else None,
                                  new, q, k, v, table, lens, parents, count, out, lse, ws, wsb,
                                  None)


@pytest.mark.parametrize("call", [window, tree])
def test_common_refusals(lib, call):
    d = pages()
    for kw, want in BAD_DIMS:
        assert call(lib, pages(**kw), opts()) == want, kw
    assert call(lib, d, None) == NULL
    assert call(lib, d, opts(), new=0) == SHAPE
    assert call(lib, d, opts(), new=65) == UNSUPPORTED
    for name in ("q", "k", "v", "table", "lens", "out", "ws"):
        assert call(lib, d, opts(), **{name: None}) == NULL, name
    for name in ("q", "k", "v", "out", "ws"):
        assert call(lib, d, opts(), **{name: ODD}) == ALIGNMENT, name
    for name in ("table", "lens", "lse"):
        assert call(lib, d, opts(), **{name: ODD2}) == ALIGNMENT, name
    assert call(lib, d, opts(), wsb=300) == WORKSPACE
    assert call(lib, d, opts(softcap=-1.0)) == SHAPE
    assert call(lib, d, opts(slopes=ODD2.value)) == ALIGNMENT
    assert call(lib, d, opts(prefix=P.value)) == UNSUPPORTED


def test_window_sizes(lib):
    assert window(lib, pages(), opts(), window=0) == SHAPE
    assert window(lib, pages(), opts(), window=-5) == SHAPE
    assert window(lib, pages(), opts(), sinks=-1) == SHAPE


def test_tree_arguments(lib):
    d, n = pages(), ctypes.c_size_t(0)
    assert tree(lib, d, opts(causal=0)) == UNSUPPORTED
    assert tree(lib, d, opts(), parents=None) == NULL
    assert tree(lib, d, opts(), parents=ODD2) == ALIGNMENT
    assert tree(lib, d, opts(), count=ODD2) == ALIGNMENT
    assert lib.wf_paged_tree_attn_workspace_bytes(ctypes.byref(d), 64, ctypes.byref(n)) == OK
    assert tree(lib, d, opts(), new=64, wsb=n.value - 1) == WORKSPACE
    assert lib.wf_paged_tree_attn_workspace_bytes(ctypes.byref(d), 0, ctypes.byref(n)) == SHAPE
    assert lib.wf_paged_tree_attn_workspace_bytes(ctypes.byref(d), 65,
                                                  ctypes.byref(n)) == UNSUPPORTED
    assert lib.wf_paged_tree_attn_workspace_bytes(ctypes.byref(d), 1, None) == NULL


def test_binding():
    x = torch.zeros((1, 4, 2, 64))
    cache, i = {"K": x, "V": x}, torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):
        bd.paged_window_attn(x, cache, i[None], i, 5)
    with pytest.raises(ValueError):
        bd.paged_tree_attn(x, cache, i[None], i, i[None])
    for n, least in ((0, 1), (-1, 0), (-2 ** 32 + 5, 0)):
        with pytest.raises(ValueError):
            bd._reach(n, "window", least)
    assert bd._reach(2 ** 32 + 1, "window", 1) == 2 ** 31 - 1    # all of it, not one
    assert bd._reach(7, "window", 1) == 7

"""Host-side refusals of paged calls at the ends of their sizes (no launch here)."""

import ctypes
import os

import pytest

from test_abi_dense import ALIGNMENT, NULL, ODD2, OK, P, UNSUPPORTED, WORKSPACE, opts, pages
from test_abi_paged_masks import tree, window
from wavelet_guided_sparse_gb300 import binding as bd


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(bd.LIB_PATH):
        from wavelet_guided_sparse_gb300 import build
        build.build()
    return bd.lib()


@pytest.mark.parametrize("call", [window, tree])
@pytest.mark.parametrize("table_pages,dtype,new,refused", [
    (262143, 1, 1, True),      # (524286 tiles of 64 keys + 2) x 4096 sequences > 2^31 - 1
    (262143, 1, 64, True),
    (262143, 0, 64, False),    # tiles of 128 keys
    (262142, 1, 1, False)])    # (524284 + 2) x 4096
def test_tiles_and_pads_fit_32_bits(lib, call, table_pages, dtype, new, refused):
    d = pages(n_seqs=4096, table_pages=table_pages, page_size=128, n_pages=10, kv_heads=1,
              q_heads=1, head_dim=64, dtype=dtype)
    n = ctypes.c_size_t(0)
    assert lib.wf_paged_attn_workspace_bytes(ctypes.byref(d), new, ctypes.byref(n)) == OK
    assert call(lib, d, opts(), new=new, wsb=0) == (UNSUPPORTED if refused else WORKSPACE)


def test_reserve_from(lib):
    d = pages()
    n = ctypes.c_size_t(0)
    assert lib.wf_pages_workspace_bytes(ctypes.byref(d), 0, 0, ctypes.byref(n)) == OK

    def call(dims=d, start=P, rows=P, refs=P, table=P, ws=P, wsb=1 << 40):
        return lib.wf_paged_reserve_from(ctypes.byref(dims), start, rows, refs, table, ws, wsb, None)

    for name in ("rows", "refs", "table", "ws"):
        assert call(**{name: None}) == NULL
    for name in ("start", "rows", "refs", "table", "ws"):
        assert call(**{name: ODD2}) == ALIGNMENT
    assert call(start=None, wsb=n.value - 1) == WORKSPACE
    assert call(pages(page_size=48)) == UNSUPPORTED

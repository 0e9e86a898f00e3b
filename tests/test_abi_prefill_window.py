"""Host-side refusals of the windowed packed-prompt attention (no launch here)."""

import ctypes
import os

import pytest
import torch

from test_abi_dense import ALIGNMENT, NULL, ODD, ODD2, OK, P, SHAPE, UNSUPPORTED, WORKSPACE, opts
from wavelet_guided_sparse_gb300 import binding as bd


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(bd.LIB_PATH):
        from wavelet_guided_sparse_gb300 import build
        build.build()
    return bd.lib()


def call(lib, o, window=10, sinks=0, q=P, qs=1024, k=P, ks=256, v=P, vs=256, cuq=P, cuk=P, out=P,
         lse=None, ws=None, wsb=0, **kw):
    base = dict(rows_q=10, rows_k=10, n_docs=2, q_heads=8, kv_heads=2, head_dim=128, dtype=0)
    d = bd.PrefillDims(**{**base, **kw})
    return lib.wf_prefill_window_attn(ctypes.byref(d), ctypes.byref(o) if o is not None else None,
                                      window, sinks, q, qs, k, ks, v, vs, cuq, cuk, out, lse, ws,
                                      wsb, None)


def test_refusals(lib):
    assert call(lib, None) == NULL
    assert call(lib, opts(), rows_q=0) == OK
    assert call(lib, opts(), window=0) == SHAPE
    assert call(lib, opts(), window=-1) == SHAPE
    assert call(lib, opts(), sinks=-1) == SHAPE
    assert call(lib, opts(prefix=P.value)) == UNSUPPORTED
    for kw, want in ((dict(rows_q=-1), SHAPE), (dict(n_docs=0), SHAPE), (dict(q_heads=9), SHAPE),
                     (dict(head_dim=32), UNSUPPORTED), (dict(rows_q=(1 << 26) + 1), UNSUPPORTED)):
        assert call(lib, opts(), **kw) == want, kw
    for name in ("q", "k", "v", "cuq", "cuk", "out"):
        assert call(lib, opts(), **{name: None}) == NULL, name
    for name in ("qs", "ks", "vs"):
        assert call(lib, opts(), **{name: 100}) == SHAPE, name
    for name in ("q", "k", "v", "out"):
        assert call(lib, opts(), **{name: ODD}) == ALIGNMENT, name
    for name in ("cuq", "cuk", "lse"):
        assert call(lib, opts(), **{name: ODD2}) == ALIGNMENT, name
    assert call(lib, opts(), ws=P, wsb=8) == WORKSPACE
    assert call(lib, opts(softcap=-0.5)) == SHAPE


def test_binding():
    x, i = torch.zeros((4, 2, 64)), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        bd.prefill_window_attn(x, x, x, i, 5)

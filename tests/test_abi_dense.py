"""Host-side refusals of the paged cache and dense attention entry points: bad
arguments are turned down before anything reaches the GPU (no launch here)."""

import ctypes
import math
import os

import pytest
import torch

from wavelet_guided_sparse_gb300 import binding as bd

OK, NULL, SHAPE, UNSUPPORTED, WORKSPACE, ALIGNMENT = 0, 1, 2, 3, 4, 7
P = ctypes.c_void_p(1 << 20)          # aligned, never dereferenced
ODD = ctypes.c_void_p((1 << 20) + 8)
ODD2 = ctypes.c_void_p((1 << 20) + 2)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(bd.LIB_PATH):
        from wavelet_guided_sparse_gb300 import build
        build.build()
    return bd.lib()


def pages(**kw):
    base = dict(n_seqs=4, q_heads=8, kv_heads=2, head_dim=128, page_size=16, n_pages=100,
                table_pages=20, dtype=0)
    base.update(kw)
    return bd.PageDims(**base)


def opts(**kw):
    base = dict(scale=0.0, softcap=0.0, causal=1, prefix=None, slopes=None)
    base.update(kw)
    return bd.AttnOpts(**base)


def test_rope_inv_freq(lib):
    f = list(bd.rope_inv_freq(64, 500000.0))
    assert len(f) == 32
    for i, x in enumerate(f):
        assert abs(x / 500000.0 ** (-2 * i / 64) - 1) < 1e-14
    out = (ctypes.c_double * 64)()
    assert lib.wf_rope_inv_freq(64, 10000.0, None) == NULL
    for r, base in ((8, 1e4), (0, 1e4), (144, 1e4), (40, 1e4), (64, 1.0), (64, math.inf),
                    (64, math.nan)):
        assert lib.wf_rope_inv_freq(r, base, out) == UNSUPPORTED


BAD_DIMS = [(dict(head_dim=96), UNSUPPORTED), (dict(dtype=2), UNSUPPORTED),
            (dict(q_heads=7), SHAPE), (dict(q_heads=0), SHAPE), (dict(kv_heads=0), SHAPE),
            (dict(n_seqs=0), SHAPE), (dict(n_pages=0), SHAPE), (dict(table_pages=0), SHAPE),
            (dict(page_size=4), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED),
            (dict(page_size=512), UNSUPPORTED), (dict(n_seqs=4097), UNSUPPORTED),
            (dict(n_pages=1 << 27), UNSUPPORTED), (dict(table_pages=1 << 28), UNSUPPORTED),
            (dict(n_seqs=4096, table_pages=1 << 24), UNSUPPORTED)]


@pytest.mark.parametrize("kw,want", BAD_DIMS)
def test_page_dims(lib, kw, want):
    n = ctypes.c_size_t(0)
    assert lib.wf_paged_attn_workspace_bytes(ctypes.byref(pages(**kw)), 1, ctypes.byref(n)) == want
    assert append(lib, pages(**kw)) == want


def test_paged_workspace(lib):
    n = ctypes.c_size_t(0)
    d = pages()
    assert lib.wf_paged_attn_workspace_bytes(ctypes.byref(d), 1, ctypes.byref(n)) == OK
    assert n.value > 256
    assert lib.wf_paged_attn_workspace_bytes(ctypes.byref(d), 0, ctypes.byref(n)) == SHAPE
    assert lib.wf_paged_attn_workspace_bytes(ctypes.byref(d), 65, ctypes.byref(n)) == UNSUPPORTED
    assert lib.wf_paged_attn_workspace_bytes(ctypes.byref(d), 1, None) == NULL
    assert lib.wf_paged_attn_workspace_bytes(None, 1, ctypes.byref(n)) == NULL


def append(lib, dims, rows=5, q=P, qs=1024, k=P, ks=256, v=P, vs=256, cu=P, held=P, pos=None,
           table=P, freq="default", rotary=128, kp=P, vp=P, qo=P, ko=None, ws=None, wsb=0):
    f = (ctypes.c_double * 64)(*[0.5] * 64) if freq == "default" else freq
    return lib.wf_paged_append(ctypes.byref(dims) if dims is not None else None, rows, q, qs, k,
                               ks, v, vs, cu, held, pos, table, f, rotary, 0, kp, vp, qo, ko, ws,
                               wsb, None)


def test_append_refusals(lib):
    d = pages()
    assert append(lib, None) == NULL
    assert append(lib, d, rows=0) == OK                    # nothing to do, nothing launched
    assert append(lib, d, rows=-1) == SHAPE
    for rotary in (-16, 8, 40, 144):
        assert append(lib, d, rotary=rotary) == SHAPE
    for name in ("k", "v", "cu", "held", "table", "kp", "vp", "freq", "q", "qo"):
        assert append(lib, d, **{name: None}) == NULL, name
    for kw in (dict(qs=1023), dict(qs=1028), dict(ks=255), dict(vs=252), dict(ks=-256)):
        assert append(lib, d, **kw) == SHAPE, kw
    for name in ("q", "k", "v", "kp", "vp", "qo", "ko"):
        assert append(lib, d, **{name: ODD}) == ALIGNMENT, name
    for name in ("cu", "held", "pos", "table"):
        assert append(lib, d, **{name: ODD2}) == ALIGNMENT, name
    assert append(lib, d, ws=P, wsb=255) == WORKSPACE
    bad = (ctypes.c_double * 64)(*[math.inf] * 64)
    assert append(lib, d, freq=bad) == SHAPE


def paged(lib, dims, o, new=1, q=P, k=P, v=P, table=P, lens=P, out=P, lse=None, ws=P,
          wsb=1 << 40):
    return lib.wf_paged_attn(ctypes.byref(dims), ctypes.byref(o) if o is not None else None, new,
                             q, k, v, table, lens, out, lse, ws, wsb, None)


def test_paged_refusals(lib):
    d = pages()
    assert paged(lib, d, None) == NULL
    assert paged(lib, d, opts(), new=0) == SHAPE
    assert paged(lib, d, opts(), new=65) == UNSUPPORTED
    for name in ("q", "k", "v", "table", "lens", "out", "ws"):
        assert paged(lib, d, opts(), **{name: None}) == NULL, name
    for name in ("q", "k", "v", "out", "ws"):
        assert paged(lib, d, opts(), **{name: ODD}) == ALIGNMENT, name
    for name in ("table", "lens", "lse"):
        assert paged(lib, d, opts(), **{name: ODD2}) == ALIGNMENT, name
    assert paged(lib, d, opts(), wsb=300) == WORKSPACE
    for kw in (dict(softcap=-1.0), dict(softcap=math.nan), dict(scale=math.inf), dict(scale=-1.0),
               dict(scale=3e38), dict(softcap=3e38), dict(scale=2.0, softcap=1e-39)):
        assert paged(lib, d, opts(**kw)) == SHAPE, kw
    assert paged(lib, d, opts(prefix=ODD2.value)) == ALIGNMENT
    assert paged(lib, d, opts(slopes=ODD2.value)) == ALIGNMENT


def prefill(lib, o, dims=None, q=P, qs=1024, k=P, ks=256, v=P, vs=256, cuq=P, cuk=P, out=P,
            lse=None, ws=None, wsb=0, **kw):
    base = dict(rows_q=10, rows_k=10, n_docs=2, q_heads=8, kv_heads=2, head_dim=128, dtype=0)
    base.update(kw)
    d = bd.PrefillDims(**base)
    return lib.wf_prefill_attn(ctypes.byref(d), ctypes.byref(o) if o is not None else None, q, qs,
                               k, ks, v, vs, cuq, cuk, out, lse, ws, wsb, None)


def test_prefill_refusals(lib):
    assert prefill(lib, None) == NULL
    assert prefill(lib, opts(), rows_q=0) == OK
    for kw, want in ((dict(rows_q=-1), SHAPE), (dict(rows_k=-1), SHAPE), (dict(n_docs=0), SHAPE),
                     (dict(q_heads=9), SHAPE), (dict(head_dim=32), UNSUPPORTED),
                     (dict(dtype=3), UNSUPPORTED), (dict(rows_q=(1 << 26) + 1), UNSUPPORTED),
                     (dict(n_docs=(1 << 20) + 1), UNSUPPORTED), (dict(q_heads=65536), UNSUPPORTED)):
        assert prefill(lib, opts(), **kw) == want, kw
    for name in ("q", "k", "v", "cuq", "cuk", "out"):
        assert prefill(lib, opts(), **{name: None}) == NULL, name
    for name in ("qs", "ks", "vs"):
        assert prefill(lib, opts(), **{name: 100}) == SHAPE, name
        assert prefill(lib, opts(), **{name: 1028}) == SHAPE, name
    for name in ("q", "k", "v", "out"):
        assert prefill(lib, opts(), **{name: ODD}) == ALIGNMENT, name
    for name in ("cuq", "cuk", "lse"):
        assert prefill(lib, opts(), **{name: ODD2}) == ALIGNMENT, name
    assert prefill(lib, opts(), ws=P, wsb=8) == WORKSPACE
    assert prefill(lib, opts(softcap=-0.5)) == SHAPE


def test_binding_refuses_cpu_tensors():
    x = torch.zeros((4, 2, 64))
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        bd.prefill_attn(x, x, x, i)
    with pytest.raises(ValueError):
        bd.paged_append(x, x, {"K": x[None], "V": x[None]}, i[None], i, i)
    with pytest.raises(ValueError):
        bd.paged_attn(x[None], {"K": x[None], "V": x[None]}, i[None], i)

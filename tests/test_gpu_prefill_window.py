"""GPU checks of the packed-prompt attention over a sliding window against
64-bit references, through the public entry point.  Rows no result may depend on
hold NaN or infinities."""

import math

import numpy as np
import pytest
import torch

from dense_common import check, f64
from mask_common import attend_masked, window_mask
from wavelet_guided_sparse_gb300 import binding as bd

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def randn(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def slope_list(hq):
    return torch.tensor([2.0 ** (-8 * (h + 1) / hq) for h in range(hq)], device="cuda")


def offsets(lens):
    return i32([0] + list(np.cumsum(lens)))


def run(dtype, d, hq, hkv, lens, window, sinks, causal, cap=0.0, bias=False, n_k=None, seed=0,
        scale=None, spare=2):
    n_k = n_k or lens
    t, tk = sum(lens) + spare, sum(n_k) + spare
    fused = randn((t, hq + 3, d), dtype, seed, 2.0)       # strided rows
    q, k, v = fused[:, :hq], randn((tk, hkv, d), dtype, seed + 1), randn((tk, hkv, d), dtype, seed + 2)
    fused[:, hq:] = math.nan
    q[sum(lens):], k[sum(n_k):], v[sum(n_k):] = math.nan, math.nan, math.inf
    masks = [window_mask(b - a + np.arange(a), b, window, sinks, causal)
             for a, b in zip(lens, n_k)]
    at = 0
    for m, n in zip(masks, n_k):                          # keys that no query sees
        k[at:at + n][torch.from_numpy(~m.any(0)).cuda()] = math.nan
        at += n
    slopes = slope_list(hq) if bias else None
    out = torch.full((t, hq, d), 7.0, dtype=dtype, device="cuda")
    ws = bd.alloc_status_workspace("cuda")
    o, lse = bd.prefill_window_attn(q, k, v, offsets(lens), window, cu_k=offsets(n_k), sinks=sinks,
                                    causal=causal, softcap=cap, slopes=slopes, scale=scale,
                                    out=out, with_lse=True, ws=ws)
    assert bd.read_device_status(ws) == 0
    assert (o[sum(lens):] == 7).all()
    qa, ka = 0, 0
    for s, (a, b, m) in enumerate(zip(lens, n_k, masks)):
        dist = np.abs((b - a + np.arange(a))[:, None] - np.arange(b)[None])
        ro, rl, ob, lb = attend_masked(f64(q[qa:qa + a]), f64(k[ka:ka + b]), f64(v[ka:ka + b]),
                                       dtype, m, dist, cap,
                                       None if slopes is None else slopes.cpu().numpy(), scale)
        check(f64(lse[qa:qa + a]), rl, lb, f"lse of sequence {s}")
        check(f64(o[qa:qa + a]), ro, ob, f"O of sequence {s}")
        qa, ka = qa + a, ka + b
    return o, lse


CASES = [
    # dtype, d, hq, hkv, lens, window, sinks, causal, cap, bias, n_k
    (BF, 128, 4, 2, [1, 2, 0, 130, 700], 100, 4, True, 0.0, False, None),
    (BF, 128, 4, 2, [1500], 1, 0, True, 0.0, False, None),                 # itself only
    (BF, 64, 3, 1, [900, 257, 300], 256, 17, True, 0.0, False, None),      # row blocks in pairs
    (BF, 128, 5, 5, [1000, 129], 130, 1, False, 0.0, False, None),
    (BF, 128, 2, 1, [1111], 128, 128, True, 30.0, False, None),
    (BF, 64, 2, 2, [1300, 64], 300, 200, False, 20.0, True, None),
    (BF, 128, 4, 1, [1024, 700], 64, 5, True, 0.0, True, None),
    (BF, 128, 6, 3, [2000], 500, 40, True, 50.0, True, None),
    (BF, 64, 4, 4, [600], 10 ** 12, 0, True, 0.0, False, None),            # all of it
    (BF, 64, 2, 1, [600], 3, 10 ** 12, True, 0.0, False, None),
    (BF, 128, 4, 2, [100, 40, 300], 90, 3, True, 0.0, False, [1000, 40, 301]),  # later rows
    (BF, 64, 2, 1, [300, 200], 50, 3, True, 0.0, False, [120, 0]),         # rows before any key
    (BF, 64, 2, 1, [300, 130], 50, 2, False, 0.0, True, [120, 1]),         # rows without a key
    (F32, 64, 2, 2, [1500], 256, 4, False, 0.0, False, None),
    (F32, 128, 4, 1, [1, 0, 333, 70], 65, 64, True, 30.0, True, None),
    (F32, 64, 6, 3, [500, 129], 64, 0, True, 0.0, True, None),
    (F32, 128, 2, 1, [50, 300], 100, 9, False, 25.0, False, [400, 20]),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_prompts(case):
    *args, n_k = CASES[case]
    run(*args, n_k=n_k, seed=case)


@pytest.mark.parametrize("window", [1, 2, 127, 128, 129, 255, 256, 257, 385])
@pytest.mark.parametrize("sinks", [0, 1, 16, 127, 128, 129, 256, 260])
def test_edges_against_tiles(window, sinks):
    for hq in (1, 2):                                     # row blocks, heads in pairs
        run(BF, 64, hq, 1, [1, 128, 129, 640, 700], window, sinks, True, seed=window + sinks)
    run(BF, 64, 2, 1, [129, 640], window, sinks, False, seed=window + sinks, bias=True)
    run(F32, 64, 2, 1, [129, 450], window, sinks, True, seed=window + sinks)


def test_window_over_everything_is_the_plain_attention():
    q, k, v = (randn((800, h, 128), BF, s) for s, h in ((1, 4), (2, 2), (3, 2)))
    cu = offsets([500, 300])
    for causal in (True, False):
        a = bd.prefill_attn(q, k, v, cu, causal=causal, with_lse=True)
        b = bd.prefill_window_attn(q, k, v, cu, 500, sinks=2, causal=causal, with_lse=True)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_rows_agree_with_the_paged_form():
    """A prompt's last rows, by the packed form and over pages."""
    n, hq, hkv, d, page = 1000, 8, 2, 128, 16
    q, k, v = (randn((n, h, d), BF, s) for s, h in ((1, hq), (2, hkv), (3, hkv)))
    cache = bd.alloc_paged_cache(64, hkv, page, d, BF, "cuda")
    table = torch.randperm(64, device="cuda").to(torch.int32)[None].contiguous()
    bd.paged_append(k, v, cache, table, i32([0, n]), i32([0]))
    for causal in (True, False):
        a, la = bd.prefill_window_attn(q, k, v, i32([0, n]), 300, sinks=4, causal=causal,
                                       with_lse=True)
        b, lb = bd.paged_window_attn(q[None, -8:].contiguous(), cache, table, i32([n]), 300,
                                     sinks=4, causal=causal, with_lse=True)
        # Two results within half a step of weights and output each (2^-8, values
        # below 5, mostly averaged).
        assert (a[-8:].double() - b[0].double()).abs().max() < 4 * 2.0 ** -8 * 5
        assert (la[-8:] - lb[0]).abs().max() < 1e-4


def test_waits_that_run_out():
    q, k, v = (randn((900, 2, 128), BF, s) for s in (1, 2, 3))
    ws = bd.alloc_status_workspace("cuda")
    call = lambda: bd.prefill_window_attn(q, k, v, offsets([900]), 200, sinks=3, ws=ws)
    ref = call()
    bd.inject_wait_timeout(300)
    call()
    assert bd.read_device_status(ws) == bd.DEV_WAIT_TIMEOUT
    bd.clear_device_status(ws)
    assert torch.equal(call(), ref) and bd.read_device_status(ws) == 0


def test_captured_with_new_offsets():
    q, k, v = (randn((900, 2, 64), BF, s) for s in (1, 2, 3))
    cu, out = offsets([900, 0]), torch.zeros_like(q)
    call = lambda o=None: bd.prefill_window_attn(q, k, v, cu, 100, sinks=3, out=o)
    call(out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(out)
    for lens in ([900, 0], [300, 600], [0, 900], [1, 2]):
        cu.copy_(offsets(lens))
        out.zero_()
        graph.replay()
        assert torch.equal(out[:sum(lens)], call()[:sum(lens)])
        assert (out[sum(lens):] == 0).all()

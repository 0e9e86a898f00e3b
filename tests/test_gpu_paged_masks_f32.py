"""GPU checks of the windowed and the tree attention where the small cases do not
reach: fp32 caches of many tiles, missing pages, waits that run out and values that
are not finite, and units that are split among more CTAs than a join reads at once."""

import math

import numpy as np
import pytest
import torch

from dense_common import check, f64
from mask_common import attend_masked, tree_mask
from test_gpu_paged_masks import i32, paged, randn, random_tree, rows_of, run_tree, run_window
from wavelet_guided_sparse_gb300 import binding as bd

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
LENS = [5000, 3111, 70, 4002, 4200, 0, 2400]


@pytest.mark.parametrize("d,new,hq,hkv,page,window,sinks,causal,cap,bias", [
    (64, 1, 20, 20, 16, 3000, 4, True, 0.0, False), (64, 5, 40, 10, 8, 2500, 64, True, 20.0, True),
    (128, 16, 10, 10, 64, 2000, 200, False, 0.0, False),
    (64, 32, 24, 8, 256, 600, 1, False, 30.0, True)])
def test_window_of_many_tiles(d, new, hq, hkv, page, window, sinks, causal, cap, bias):
    run_window(F32, d, hq, hkv, page, LENS, new, window, sinks, causal, cap, bias, seed=new)


@pytest.mark.parametrize("d,nodes,hq,hkv,page,cap,bias", [
    (64, 8, 20, 20, 16, 0.0, False), (64, 20, 16, 8, 8, 20.0, True),
    (128, 33, 10, 10, 64, 0.0, True), (64, 3, 40, 10, 128, 30.0, False)])
def test_tree_of_many_tiles(d, nodes, hq, hkv, page, cap, bias):
    rng = np.random.default_rng(nodes)
    trees = [random_tree(max(1, nodes - 3 * s), rng) if n else [] for s, n in enumerate(LENS)]
    run_tree(F32, d, hq, hkv, page, LENS, nodes, trees, cap, bias, seed=nodes)


# Tiles of 64 keys (fp32, and bf16 with at most four rows a key head) or 128; a CTA a tile
# until there are no more CTAs.
@pytest.mark.parametrize("dtype,d,hq,nodes,tile", [
    (BF, 64, 2, 20, 128), (BF, 128, 4, 9, 128), (BF, 128, 4, 64, 128), (BF, 64, 2, 2, 64),
    (BF, 128, 1, 4, 64), (F32, 64, 2, 3, 64), (F32, 128, 2, 20, 64)])
@pytest.mark.parametrize("tiles", [31, 32, 33, 34, 65, 200])
def test_units_in_many_parts(dtype, d, hq, nodes, tile, tiles):
    """One sequence and one key head: 33 parts and more, which the join reads 32 at a time."""
    n = tiles * tile - 7
    tree = random_tree(nodes, np.random.default_rng(tiles))
    run_tree(dtype, d, hq, 1, 16, [n], nodes, [tree], 0.0, False, seed=tiles)
    run_window(dtype, d, hq, 1, 16, [n], nodes, n - 5, 2, True, 0.0, True, seed=tiles + 1)


@pytest.mark.parametrize("new,hq,hkv", [(1, 4, 2), (20, 8, 2)])
def test_waits_that_run_out(new, hq, hkv):
    cache, table = paged([900, 300], 16, hkv, 128, F32, 13)
    t, q = i32(table.tolist()), randn((2, new, hq, 128), F32, 2)
    tree = i32([random_tree(new, np.random.default_rng(new))] * 2)
    lens, wt = i32([900, 300]), bd.alloc_paged_tree_workspace(q, cache, t)
    ww = bd.alloc_paged_attn_workspace(q, cache, t)
    for ws, call in ((wt, lambda: bd.paged_tree_attn(q, cache, t, lens, tree, wt)),
                     (ww, lambda: bd.paged_window_attn(q, cache, t, lens, 250, ww, sinks=70))):
        ref = call()
        bd.inject_wait_timeout(300)
        call()
        assert bd.read_device_status(ws) == bd.DEV_WAIT_TIMEOUT
        bd.clear_device_status(ws)
        assert torch.equal(call(), ref) and bd.read_device_status(ws) == 0


@pytest.mark.parametrize("nodes,hq,hkv", [(4, 4, 2), (30, 8, 2)])
def test_tree_over_missing_pages(nodes, hq, hkv):
    n, page = 1000, 16
    cache, table = paged([n], page, hkv, 64, F32, 17)
    keep = np.ones(n, bool)
    for e in (3, 20, 21, 22, 23, 40):
        table[0, e] = 10 ** 6 if e % 2 else -5
        keep[e * page:(e + 1) * page] = False
    tree = random_tree(nodes, np.random.default_rng(3))
    q, t = randn((1, nodes, hq, 64), F32, 4), i32(table.tolist())
    ws = bd.alloc_paged_tree_workspace(q, cache, t)
    for _ in range(2):                                # stale stages of the first hold values
        o, lse = bd.paged_tree_attn(q, cache, t, i32([n]), i32([tree]), ws, with_lse=True)
        assert bd.read_device_status(ws) == bd.DEV_BAD_INDEX
        k, v = rows_of(cache, np.where((table < 0) | (table > 10 ** 5), 0, table), 0, n)
        ro, rl, ob, lb = attend_masked(f64(q[0]), k, v, F32, tree_mask(n - nodes, tree)[0] & keep)
        check(f64(lse[0]), rl, lb, "lse")
        check(f64(o[0]), ro, ob, "O")


@pytest.mark.parametrize("nodes,hq,hkv", [(8, 4, 2), (24, 8, 2)])
def test_visible_nans_and_infinities_show_and_hidden_ones_do_not(nodes, hq, hkv):
    n, d = 700, 128
    tree = [-1, 0, 1, -1] + [3] * (nodes - 4)
    cache, table = paged([n], 16, hkv, d, F32, 21)
    t, q = i32(table.tolist()), randn((1, nodes, hq, d), F32, 22).abs()
    at = lambda row: (int(table[0, row // 16]), slice(None), row % 16)
    base = n - nodes
    cache["K"][at(base + 1)] = math.nan                 # node 1: seen by nodes 1 and 2
    cache["V"][at(base + 3) + (5,)] = math.inf          # node 3: seen by itself and 4..
    cache["K"][at(300)] = -math.inf                     # all rows: weight 0
    o, lse = bd.paged_tree_attn(q, cache, t, i32([n]), i32([tree]), with_lse=True)
    bad = torch.zeros(nodes, dtype=torch.bool, device="cuda")
    bad[1:3] = True
    assert lse[0, bad].isnan().all() and lse[0, ~bad].isfinite().all()
    assert o[0, bad].isnan().all()
    assert (o[0, 3:, :, 5] == math.inf).all()
    assert o[0, ~bad][:, :, 6:].isfinite().all() and o[0, ~bad][:, :, :5].isfinite().all()
    w = bd.paged_window_attn(q[:, :4].contiguous(), cache, t, i32([base]), 200)
    assert w.isfinite().all()
    w = bd.paged_window_attn(q[:, :4].contiguous(), cache, t, i32([base + 3]), 100)
    assert w[0, 3].isnan().all() and w[0, :2].isfinite().all()


@pytest.mark.parametrize("seqs,every", [(129, 1), (300, 3), (4096, 61), (1000, 997)])
@pytest.mark.parametrize("dtype,hq,nodes", [(BF, 2, 2), (BF, 4, 6), (F32, 2, 3)])
def test_live_sequences_far_apart(dtype, hq, nodes, seqs, every):
    """Units are found past blocks of sequences, idle ones and whole idle blocks among them."""
    rng = np.random.default_rng(seqs + nodes)
    at = [s for s in range(seqs) if s % every == every // 2]
    lens = [0] * seqs
    for s in at:
        lens[s] = int(rng.integers(nodes, 200))
    trees = [random_tree(int(rng.integers(1, nodes + 1)), rng) if n else [] for n in lens]
    run_tree(dtype, 64, hq, 2, 8, lens, nodes, trees, 0.0, False, seed=seqs)
    run_window(dtype, 64, hq, 2, 8, lens, nodes, 40, 3, True, 0.0, False, seed=seqs + 1)

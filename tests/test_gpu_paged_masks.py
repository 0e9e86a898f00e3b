"""GPU checks of the paged attention over a sliding window and by drafted trees
against 64-bit references, through the public entry points.  Rows no result may
depend on hold NaN or infinities."""

import math

import numpy as np
import pytest
import torch

from dense_common import check, f64
from mask_common import attend_masked, tree_mask, window_mask
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


def paged(lens, page, hkv, d, dtype, seed, needed=None):
    """A cache in shuffled pages.  needed[s] [n]: rows that some query sees; pages
    without one have no entry, and rows behind the end hold NaN and infinities."""
    rng = np.random.default_rng(seed)
    need = [-(-n // page) for n in lens]
    order, at = rng.permutation(sum(need) + 2), 0
    table = np.full((len(lens), max(max(need), 1)), -7)
    live = np.zeros((sum(need) + 2, page), bool)
    for s, n in enumerate(lens):
        for e in range(need[s]):
            rows = min(page, n - e * page)
            if needed is None or needed[s][e * page:e * page + rows].any():
                table[s, e] = order[at]
                live[order[at], :rows] = True
            at += 1
    cache = {"K": randn((len(order), hkv, page, d), dtype, seed + 1),
             "V": randn((len(order), hkv, page, d), dtype, seed + 2)}
    dead = ~torch.from_numpy(live).cuda()[:, None, :, None]
    cache["K"].masked_fill_(dead, math.nan)
    cache["V"].masked_fill_(dead, math.inf)
    return cache, table


def rows_of(cache, table, s, n):
    page = cache["K"].shape[2]
    out = []
    for name in ("K", "V"):
        x = f64(cache[name])
        x = np.concatenate([x[max(p, 0)] for p in table[s, :-(-n // page)]], 1)[:, :n] if n else \
            np.zeros((x.shape[1], 0, x.shape[3]))
        out.append(x.transpose(1, 0, 2))
    return out


# ------------------------------------------------------------------ window
def run_window(dtype, d, hq, hkv, page, lens, new, window, sinks, causal, cap, bias, seed=0):
    masks = [window_mask(n - new + np.arange(new), n, window, sinks, causal) for n in lens]
    cache, table = paged(lens, page, hkv, d, dtype, seed, [m.any(0) for m in masks])
    q = randn((len(lens), new, hq, d), dtype, seed + 3, 2.0)
    slopes = slope_list(hq) if bias else None
    ws = bd.alloc_paged_attn_workspace(q, cache, i32(table.tolist()))
    o, lse = bd.paged_window_attn(q, cache, i32(table.tolist()), i32(lens), window, ws, sinks=sinks,
                                  causal=causal, softcap=cap, slopes=slopes, with_lse=True)
    assert bd.read_device_status(ws) == 0
    for s, n in enumerate(lens):
        k, v = rows_of(cache, table, s, n)
        dist = np.abs((n - new + np.arange(new))[:, None] - np.arange(n)[None])
        ro, rl, ob, lb = attend_masked(f64(q[s]), k, v, dtype, masks[s], dist, cap,
                                       None if slopes is None else slopes.cpu().numpy())
        check(f64(lse[s]), rl, lb, f"lse of sequence {s}")
        check(f64(o[s]), ro, ob, f"O of sequence {s}")
    return o, lse, (q, cache, i32(table.tolist()), i32(lens), ws)


WINDOWS = [
    # dtype, d, hq, hkv, page, lens, new, window, sinks, causal, cap, bias
    (BF, 128, 32, 8, 16, [1, 17, 64, 65, 0, 1000, 3001], 1, 100, 4, True, 0.0, False),
    (BF, 128, 32, 8, 16, [1000, 63], 1, 1, 0, True, 0.0, False),          # itself only
    (BF, 128, 8, 2, 8, [900, 130, 129, 128], 1, 64, 64, True, 0.0, False),
    (BF, 128, 4, 4, 64, [63, 129, 700], 5, 128, 1, False, 20.0, True),
    (BF, 64, 12, 4, 8, [5, 900, 31], 5, 33, 9, True, 0.0, True),
    (BF, 128, 2, 2, 256, [64, 70, 4097], 64, 500, 300, True, 0.0, False),
    (BF, 64, 6, 2, 16, [500, 90], 32, 7, 20, False, 0.0, False),          # 96 rows: two blocks
    (BF, 128, 8, 2, 64, [600, 64, 33, 0], 64, 40, 0, True, 30.0, True),   # four blocks
    (BF, 64, 1, 1, 8, [3, 2], 8, 4, 2, True, 0.0, False),                 # rows before any key
    (BF, 64, 1, 1, 8, [3, 2], 8, 4, 1, False, 0.0, False),                # rows without a key
    (BF, 64, 130, 1, 16, [700, 40], 2, 100, 3, True, 0.0, True),          # 130 heads a key head
    (BF, 128, 6, 6, 16, [300, 0, 65], 3, 70, 2, True, 30.0, True),        # three rows a key head
    (BF, 128, 16, 1, 128, [2000], 1, 10 ** 12, 5, True, 0.0, False),      # all of it
    (BF, 128, 4, 1, 32, [2000, 40], 2, 300, 10 ** 12, True, 0.0, False),
    (F32, 64, 2, 2, 32, [1056, 4000], 32, 256, 64, False, 0.0, False),
    (F32, 128, 4, 1, 16, [1, 0, 1333], 1, 200, 4, True, 30.0, True),
    (F32, 128, 8, 2, 8, [500, 77, 0, 6], 5, 64, 3, True, 0.0, False),
    (F32, 128, 4, 1, 8, [333, 20], 16, 90, 70, True, 25.0, True),         # 64 rows
    (F32, 64, 9, 3, 8, [700, 41], 4, 30, 0, False, 0.0, True),
]


@pytest.mark.parametrize("args", WINDOWS)
def test_window(args):
    run_window(*args, seed=WINDOWS.index(args))


@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 127, 128, 129, 191, 193])
@pytest.mark.parametrize("sinks", [0, 1, 63, 64, 65, 128])
def test_window_edges_against_tiles(window, sinks):
    run_window(BF, 64, 2, 1, 8, [n for n in (1, 64, 128, 129, 192, 193, 320, 321, 450)], 3, window,
               sinks, True, 0.0, False, seed=window + sinks)


@pytest.mark.parametrize("new,hq,hkv,page,window,sinks,causal,cap,bias", [
    (32, 40, 10, 16, 5000, 4, False, 0.0, False), (64, 32, 8, 64, 3000, 200, True, 0.0, True),
    (5, 60, 15, 8, 4000, 64, True, 20.0, True), (1, 32, 8, 128, 6000, 130, True, 0.0, False),
    (64, 40, 10, 256, 1000, 1, False, 30.0, False)])
def test_window_of_many_tiles(new, hq, hkv, page, window, sinks, causal, cap, bias):
    """Some tens of key tiles a CTA, in parts of several units."""
    run_window(BF, 64, hq, hkv, page, [9000, 7111, 70, 5002, 8200, 0, 6400], new, window, sinks,
               causal, cap, bias, seed=new)


@pytest.mark.parametrize("new,hq,hkv", [(1, 4, 2), (20, 8, 2), (64, 16, 2)])
def test_window_waits_that_run_out(new, hq, hkv):
    cache, table = paged([900, 300], 16, hkv, 128, BF, 13)
    t, q = i32(table.tolist()), randn((2, new, hq, 128), BF, 2)
    ws = bd.alloc_paged_attn_workspace(q, cache, t)
    call = lambda: bd.paged_window_attn(q, cache, t, i32([900, 300]), 250, ws, sinks=70)
    ref = call()
    bd.inject_wait_timeout(300)
    call()
    assert bd.read_device_status(ws) == bd.DEV_WAIT_TIMEOUT
    bd.clear_device_status(ws)
    assert torch.equal(call(), ref) and bd.read_device_status(ws) == 0


def check_same(got, want, bounds, what):
    """Two results that each lie within `bounds` of the same exact ones."""
    for x, y, b, name in zip(got, want, bounds, ("O", "lse")):
        x, y = f64(x), f64(y)
        with np.errstate(invalid="ignore"):
            assert ((x == y) | (np.abs(x - y) <= 2 * b)).all(), f"{name} of {what}"


def test_window_over_everything_is_the_plain_attention():
    lens = [700, 64, 1]
    cache, table = paged(lens, 16, 2, 128, BF, 5)
    q, t, n = randn((3, 4, 8, 128), BF, 1), i32(table.tolist()), i32(lens)
    for causal in (True, False):
        a = bd.paged_attn(q, cache, t, n, causal=causal, with_lse=True)
        for sinks in (0, 3, 2000):
            b = bd.paged_window_attn(q, cache, t, n, 700, sinks=sinks, causal=causal, with_lse=True)
            for s, m in enumerate(lens):
                seen = window_mask(m - 4 + np.arange(4), m, 700, sinks, causal)
                ob, lb = attend_masked(f64(q[s]), *rows_of(cache, table, s, m), BF, seen)[2:]
                check_same([x[s] for x in b], [x[s] for x in a], (ob, lb), f"sequence {s}")


def test_window_of_released_pages():
    """A sequence that gives back what fell out of its window goes on as before."""
    page, window, sinks, n = 16, 100, 20, 900
    cache, table = paged([n, 500], page, 2, 64, BF, 7)
    t, refs = i32(table.tolist()), bd.alloc_page_refs(cache["K"].shape[0], "cuda")
    refs[t[t >= 0].long()] = 1
    t.clamp_(min=-1)
    q, lens = randn((2, 3, 4, 64), BF, 8), i32([n, 500])
    ws = bd.alloc_paged_attn_workspace(q, cache, t)
    before = bd.paged_window_attn(q, cache, t, lens, window, ws, sinks=sinks)
    bd.paged_release(cache, t, refs, i32([sinks] * 2), lens - 3 - window + 1, ws)
    # Rows 0..19 take two pages, the window's and the new rows' last 102 at most eight.
    assert ((t >= 0).sum(1) <= 10).all() and refs.sum() == (t >= 0).sum()
    gone = refs == 0
    cache["K"][gone], cache["V"][gone] = math.nan, math.nan
    after = bd.paged_window_attn(q, cache, t, lens, window, ws, sinks=sinks)
    assert torch.equal(before, after)
    assert bd.read_device_status(ws) == 0


def test_window_far_out():
    """Positions past 2^24: only the window's pages exist."""
    page, n = 256, (1 << 24) + 12345
    table = torch.full((1, n // page + 2), -1, dtype=torch.int32)
    first = (n - 300) // page
    table[0, 0], table[0, first:n // page + 1] = 0, torch.arange(1, n // page + 2 - first)
    cache = {x: randn((4, 1, page, 64), BF, i) for i, x in enumerate("KV")}
    q = randn((1, 1, 2, 64), BF, 9)
    slopes = slope_list(2)
    o, lse = bd.paged_window_attn(q, cache, table.cuda(), i32([n]), 290, sinks=5, slopes=slopes,
                                  with_lse=True)
    at = np.concatenate([np.arange(5), np.arange(n - 290, n)])
    tab = table[0].numpy()
    k, v = (np.stack([f64(cache[x])[tab[j // page], :, j % page] for j in at]) for x in "KV")
    ro, rl, ob, lb = attend_masked(f64(q[0]), k, v, BF, np.ones((1, len(at)), bool),
                                   (n - 1 - at)[None].astype(float), slopes=slopes.cpu().numpy())
    check(f64(lse[0]), rl, lb + 2.0 ** -20 * np.abs(rl), "lse")
    check(f64(o[0]), ro, ob, "O")


def test_window_flags_pages_that_are_needed_and_missing():
    cache, table = paged([300], 16, 1, 64, BF, 3)
    q = randn((1, 1, 1, 64), BF, 1)
    ws = bd.alloc_paged_attn_workspace(q, cache, i32(table.tolist()))
    table[0, 0] = -1
    bd.paged_window_attn(q, cache, i32(table.tolist()), i32([300]), 50, ws)
    assert bd.read_device_status(ws) == 0             # no query sees it
    bd.paged_window_attn(q, cache, i32(table.tolist()), i32([300]), 50, ws, sinks=1)
    assert bd.read_device_status(ws) == bd.DEV_BAD_INDEX


# ------------------------------------------------------------------ trees
def random_tree(n, rng):
    return [-1] + [int(rng.integers(-1, i)) if rng.random() < 0.5 else i - 1 for i in range(1, n)]


def run_tree(dtype, d, hq, hkv, page, lens, nodes, trees, cap, bias, seed=0, scale=None):
    """lens: rows of each sequence, its nodes' included."""
    cache, table = paged(lens, page, hkv, d, dtype, seed)
    q = randn((len(lens), nodes, hq, d), dtype, seed + 3, 2.0)
    parents = np.full((len(lens), nodes), 99)         # behind a tree: anything
    for s, t in enumerate(trees):
        parents[s, :len(t)] = t
        q[s, len(t):] = math.nan
    slopes = slope_list(hq) if bias else None
    ws = bd.alloc_paged_tree_workspace(q, cache, i32(table.tolist()))
    count = None if all(len(t) == nodes for t in trees) else i32([len(t) for t in trees])
    o, lse = bd.paged_tree_attn(q, cache, i32(table.tolist()), i32(lens), i32(parents.tolist()), ws,
                                tree_len=count, softcap=cap, slopes=slopes, scale=scale,
                                with_lse=True)
    assert bd.read_device_status(ws) == 0
    for s, (n, t) in enumerate(zip(lens, trees)):
        live = len(t) if n else 0
        k, v = rows_of(cache, table, s, n)
        assert (o[s, live:] == 0).all() and (lse[s, live:] == -math.inf).all()
        if not live:
            continue
        base = n - live
        seen, depth = tree_mask(base, t)
        at = np.concatenate([np.arange(base), base + depth])
        dist = np.abs((base + depth)[:, None] - at[None])
        ro, rl, ob, lb = attend_masked(f64(q[s, :live]), k, v, dtype, seen, dist, cap,
                                       None if slopes is None else slopes.cpu().numpy(), scale)
        check(f64(lse[s, :live]), rl, lb, f"lse of sequence {s}")
        check(f64(o[s, :live]), ro, ob, f"O of sequence {s}")
    return o, lse


RNG = np.random.default_rng(0)
CHAIN, STAR = list(range(-1, 63)), [-1] + [0] * 63
TREES = [
    # dtype, d, hq, hkv, page, lens, nodes, trees, cap, bias
    (BF, 128, 32, 8, 16, [1, 17, 300, 65], 1, [[-1]] * 4, 0.0, False),
    (BF, 128, 32, 8, 16, [9, 100, 0, 1000], 8, [random_tree(8, RNG), random_tree(5, RNG), [],
                                                random_tree(8, RNG)], 0.0, False),
    (BF, 128, 8, 2, 64, [64, 200, 4000], 64, [CHAIN, STAR, random_tree(64, RNG)], 0.0, False),
    (BF, 128, 8, 1, 8, [700, 77], 13, [random_tree(13, RNG), [-1] * 9], 30.0, True),
    (BF, 64, 4, 4, 32, [130, 129, 128, 127, 3], 3, [[-1, 0, 1], [-1, 0, 0], [-1, -1, -1],
                                                    [-1, 0], [-1, -1, 1]], 0.0, True),
    (BF, 64, 6, 2, 16, [500, 90], 26, [random_tree(26, RNG), random_tree(20, RNG)], 20.0, False),
    (BF, 128, 5, 5, 256, [1500, 600], 40, [random_tree(33, RNG), random_tree(40, RNG)], 0.0, True),
    (BF, 128, 16, 2, 128, [2000, 64], 64, [random_tree(64, RNG), CHAIN], 50.0, True),
    (BF, 128, 9, 3, 16, [333, 40, 800], 32, [random_tree(32, RNG), random_tree(32, RNG),
                                             random_tree(1, RNG)], 0.0, False),
    (BF, 64, 32, 8, 8, [100, 2500], 50, [random_tree(50, RNG), random_tree(47, RNG)], 0.0, False),
    (BF, 128, 40, 1, 16, [777], 20, [random_tree(20, RNG)], 0.0, True),   # 800 rows a key head
    (BF, 64, 130, 1, 16, [700, 40], 2, [[-1, 0], [-1, -1]], 20.0, True),  # 130 heads a key head
    (BF, 128, 6, 6, 16, [300, 0, 65], 3, [[-1, 0, 0], [], [-1, -1]], 30.0, True),  # three rows
    (F32, 64, 2, 2, 32, [1056, 13], 13, [random_tree(13, RNG), random_tree(13, RNG)], 0.0, False),
    (F32, 128, 4, 1, 16, [5, 0, 333], 5, [random_tree(5, RNG), random_tree(5, RNG),
                                          random_tree(3, RNG)], 30.0, True),
    (F32, 128, 8, 2, 8, [500, 77], 16, [random_tree(16, RNG), random_tree(16, RNG)], 0.0, True),
    (F32, 64, 9, 3, 8, [300, 64], 64, [STAR, CHAIN], 0.0, False),
]


@pytest.mark.parametrize("case", range(len(TREES)))
def test_tree(case):
    run_tree(*TREES[case], seed=100 + case)


@pytest.mark.parametrize("nodes,hq,hkv,page,bias", [
    (20, 40, 10, 16, False), (26, 32, 8, 64, True), (64, 40, 10, 128, False), (33, 60, 15, 8, True)])
def test_tree_of_many_tiles(nodes, hq, hkv, page, bias):
    """Some tens of key tiles a CTA, in parts of several units."""
    rng = np.random.default_rng(nodes)
    lens = [9000, 7111, 70, 5002, 8200, 0, 6400]
    trees = [random_tree(max(1, nodes - 3 * s), rng) if n else [] for s, n in enumerate(lens)]
    run_tree(BF, 64, hq, hkv, page, lens, nodes, trees, 0.0, bias, seed=nodes)


@pytest.mark.parametrize("hq,hkv", [(4, 4), (8, 2), (12, 4), (24, 2)])
def test_tree_edges_against_tiles(hq, hkv):
    """Trees that begin, end and lie across the borders of key tiles."""
    for nodes in (6, 33):
        rng = np.random.default_rng(nodes)
        lens = [nodes, nodes + 1, 64, 128 + nodes, 127 + nodes, 129, 192 + nodes // 2, 256, 257]
        run_tree(BF, 64, hq, hkv, 8, lens, nodes, [random_tree(nodes, rng) for _ in lens], 0.0,
                 True, seed=nodes)


@pytest.mark.parametrize("nodes", [1, 4, 40])
def test_a_chain_is_the_causal_attention(nodes):
    """A tree without branches sees what new tokens see."""
    lens = [700, 64, 41]
    cache, table = paged(lens, 16, 2, 128, BF, 5)
    q, t, n = randn((3, nodes, 8, 128), BF, 1), i32(table.tolist()), i32(lens)
    a = bd.paged_attn(q, cache, t, n, with_lse=True)
    b = bd.paged_tree_attn(q, cache, t, n, i32([list(range(-1, nodes - 1))] * 3), with_lse=True)
    for s, m in enumerate(lens):
        seen = tree_mask(m - nodes, list(range(-1, nodes - 1)))[0]
        ob, lb = attend_masked(f64(q[s]), *rows_of(cache, table, s, m), BF, seen)[2:]
        check_same([x[s] for x in b], [x[s] for x in a], (ob, lb), f"sequence {s}")


def test_tree_flags():
    cache, table = paged([100, 3, 50, 60, 0], 16, 1, 64, BF, 3)
    t, lens = i32(table.tolist()), [100, 3, 50, 60, 0]
    q = randn((5, 4, 2, 64), BF, 1)
    ws = bd.alloc_paged_tree_workspace(q, cache, t)
    tree = [[-1, 0, 0, 2]] * 5
    ref = bd.paged_tree_attn(q, cache, t, i32([100, 0, 50, 60, 0]), i32(tree), ws)
    assert bd.read_device_status(ws) == 0
    got = bd.paged_tree_attn(q, cache, t, i32(lens), i32(tree), ws)     # 3 rows, 4 nodes
    assert bd.read_device_status(ws) == bd.DEV_BAD_INDEX and torch.equal(got, ref)
    assert (got[1] == 0).all()
    for bad in (2, 5, 2 ** 31 - 1):                   # node 2's parent not before it
        bd.clear_device_status(ws)
        odd = [[-1, 0, bad, 2]] + tree[1:]
        got = bd.paged_tree_attn(q, cache, t, i32([100, 0, 50, 60, 0]), i32(odd), ws)
        assert bd.read_device_status(ws) == bd.DEV_BAD_INDEX
        want = bd.paged_tree_attn(q, cache, t, i32([100, 0, 50, 60, 0]),
                                  i32([[-1, 0, -1, 2]] + tree[1:]))
        assert torch.equal(got, want)
    bd.clear_device_status(ws)
    got = bd.paged_tree_attn(q, cache, t, i32([100, 0, 50, 60, 0]), i32(tree), ws,
                             tree_len=i32([4, 4, 5, -1, 9]))
    assert bd.read_device_status(ws) == bd.DEV_BAD_INDEX
    ref[3] = 0
    assert torch.equal(got, ref)


@pytest.mark.parametrize("nodes,hq,hkv", [(6, 4, 2), (64, 16, 2)])
def test_tree_captured_with_new_lengths(nodes, hq, hkv):
    rng = np.random.default_rng(1)
    cache, table = paged([900, 900], 16, hkv, 128, BF, 11)
    t, q = i32(table.tolist()), randn((2, nodes, hq, 128), BF, 2)
    ws = bd.alloc_paged_tree_workspace(q, cache, t)
    lens, parents, count = i32([900, 70]), i32([random_tree(nodes, rng)] * 2), i32([nodes, nodes])
    out = torch.empty_like(q)
    call = lambda **kw: bd.paged_tree_attn(q, cache, t, lens, parents, tree_len=count, **kw)
    call(ws=ws, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(ws=ws, out=out)
    for n, c in (([900, 70], [nodes, nodes]), ([65, 900], [nodes, 1]), ([0, 899], [nodes, 5])):
        lens.copy_(i32(n))
        count.copy_(i32(c))
        parents.copy_(i32([random_tree(nodes, rng) for _ in range(2)]))
        graph.replay()
        assert torch.equal(out, call())
    assert bd.read_device_status(ws) == 0


# ------------------------------------------------------------------ both
def test_visible_nans_and_infinities_show_and_hidden_ones_do_not():
    """A key that holds NaN shows in the rows that see it and in no other; an infinite
    value in its column of the rows that see it (the column's other rows meet it with
    weights of 0: values that a mask hides must be finite); a key of the opposite
    sign of infinity weighs nothing."""
    n, nodes, hq, hkv, d = 700, 24, 8, 2, 128
    tree = [-1, 0, 1, -1] + [3] * 20
    cache, table = paged([n], 16, hkv, d, BF, 21)
    t, q = i32(table.tolist()), randn((1, nodes, hq, d), BF, 22).abs()
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
    # A window that ends before them sees none of it.
    w = bd.paged_window_attn(q[:, :8].contiguous(), cache, t, i32([base]), 200)
    assert w.isfinite().all()
    w = bd.paged_window_attn(q[:, :8].contiguous(), cache, t, i32([base + 3]), 100)
    assert w[0, 7].isnan().all() and w[0, :6].isfinite().all()


@pytest.mark.parametrize("hq,hkv", [(4, 2), (2, 2)])
def test_many_sequences_with_idle_ones_between(hq, hkv):
    rng = np.random.default_rng(hq)
    lens = [int(rng.integers(0, 300)) if rng.random() < 0.6 else 0 for _ in range(150)]
    run_window(BF, 64, hq, hkv, 8, lens, 2, 70, 5, True, 0.0, False, seed=hq)
    lens = [n and max(n, 4) for n in lens]
    run_tree(BF, 64, hq, hkv, 8, lens, 4, [random_tree(int(rng.integers(1, 5)), rng) if n else []
                                           for n in lens], 0.0, False, seed=hq)


def test_two_streams_at_once():
    calls, want = [], []
    for s in range(2):
        cache, table = paged([3000, 900, 2500], 16, 4, 128, BF, 31 + s)
        t, lens = i32(table.tolist()), i32([3000, 900, 2500])
        q = randn((3, 20, 16, 128), BF, 33 + s)
        tree = i32([random_tree(20, np.random.default_rng(s + i)) for i in range(3)])
        wt = bd.alloc_paged_tree_workspace(q, cache, t)
        ww = bd.alloc_paged_attn_workspace(q, cache, t)
        calls.append(lambda stream, q=q, cache=cache, t=t, lens=lens, tree=tree, wt=wt, ww=ww: (
            bd.paged_tree_attn(q, cache, t, lens, tree, wt, stream=stream),
            bd.paged_window_attn(q, cache, t, lens, 700, ww, sinks=9, stream=stream)))
        want.append(calls[-1](None))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for s in range(2):
            got[s].append(calls[s](streams[s]))
    torch.cuda.synchronize()
    for s in range(2):
        for r in got[s]:
            assert all(torch.equal(x, y) for x, y in zip(r, want[s]))


# ------------------------------------------------------------------ a drafting step
def test_append_verify_keep():
    """Drafted tokens filed at their depths, verified, the accepted path kept: the
    cache and the next token's attention are those of the path written directly."""
    hq, hkv, d, page, old = 4, 2, 64, 16, [37, 100]
    tree = [[-1, 0, 0, 1, 2, 2], [-1, -1, 1, 2, 3, 0]]
    path = [[0, 2, 5], [1, 2, 3, 4]]
    n = len(tree[0])
    k, v, q = (randn((2 * n, h, d), BF, s) for s, h in ((1, hkv), (2, hkv), (3, hq)))
    freq = bd.rope_inv_freq(d)
    pools = []
    for way in ("tree", "direct"):
        cache = {x: randn((40, hkv, page, d), BF, 20 + i) for i, x in enumerate("KV")}
        table, refs = bd.alloc_page_table(2, 12, "cuda"), bd.alloc_page_refs(40, "cuda")
        pw = bd.alloc_pages_workspace(cache, table, max_keep=n)
        bd.paged_reserve(cache, table, refs, i32([m + n for m in old]), pw)
        if way == "tree":
            depth = [tree_mask(0, t)[1] for t in tree]
            pos = [old[s] + int(depth[s][i]) for s in range(2) for i in range(n)]
            new = bd.paged_append(k, v, cache, table, i32([0, n, 2 * n]), i32(old), q=q,
                                  inv_freq=freq, positions=i32(pos))
            lens = i32([m + n for m in old])
            seen = bd.paged_tree_attn(new["Q"].view(2, n, hq, d), cache, table, lens, i32(tree))
            bd.paged_keep(cache, table, lens, i32(old),
                          i32([[m + i for i in p] + [0] * (n - len(p))
                               for m, p in zip(old, path)]),
                          i32([len(p) for p in path]), refs, pw)
            assert bd.read_device_status(pw) == 0
        else:
            rows = [s * n + i for s in range(2) for i in path[s]]
            new = bd.paged_append(k[rows], v[rows], cache, table, i32([0, 3, 7]), i32(old),
                                  q=q[rows], inv_freq=freq)
            step = 0
            for s in range(2):                       # each prefix of the path, as one sequence
                for i, node in enumerate(path[s]):
                    one = bd.paged_attn(new["Q"][step][None, None], cache, table[s:s + 1],
                                        i32([old[s] + i + 1]))
                    err = (one[0, 0].double() - seen[s, node].double()).abs().max()
                    # Both within half a step of their own rounding, and the tree's
                    # weights rounded once more: 3 of them, of values below 4.
                    assert err < 3 * 2.0 ** -8 * 4
                    step += 1
            bd.paged_keep(cache, table, i32([m + n for m in old]),
                          i32([m + len(p) for m, p in zip(old, path)]), refs=refs, ws=pw)
        pools.append((cache, table, refs))
    (c0, t0, r0), (c1, t1, r1) = pools
    assert torch.equal(t0, t1) and torch.equal(r0, r1)
    for s, m in enumerate(m + len(p) for m, p in zip(old, path)):
        for x in "KV":
            a, b = (c[x][t[s, :-(-m // page)].long()].transpose(1, 2).flatten(0, 1)[:m]
                    for c, t in ((c0, t0), (c1, t1)))
            assert torch.equal(a, b)


@pytest.mark.parametrize("nodes,hq,hkv", [(1, 4, 2), (20, 8, 2), (64, 16, 2)])
def test_waits_that_run_out(nodes, hq, hkv):
    cache, table = paged([900, 300], 16, hkv, 128, BF, 13)
    t, q = i32(table.tolist()), randn((2, nodes, hq, 128), BF, 2)
    ws = bd.alloc_paged_tree_workspace(q, cache, t)
    tree = i32([random_tree(nodes, np.random.default_rng(nodes))] * 2)
    call = lambda: bd.paged_tree_attn(q, cache, t, i32([900, 300]), tree, ws)
    ref = call()
    bd.inject_wait_timeout(300)
    call()
    assert bd.read_device_status(ws) == bd.DEV_WAIT_TIMEOUT
    bd.clear_device_status(ws)
    assert torch.equal(call(), ref) and bd.read_device_status(ws) == 0


@pytest.mark.parametrize("nodes,hq,hkv", [(30, 8, 2), (64, 16, 2)])
def test_tree_over_missing_pages(nodes, hq, hkv):
    """Rows of pages outside the pool do not count, and nothing they left behind does."""
    n, page = 1000, 16
    cache, table = paged([n], page, hkv, 64, BF, 17)
    gone = [3, 20, 21, 22, 23, 40]
    keep = np.ones(n, bool)
    for e in gone:
        table[0, e] = 10 ** 6 if e % 2 else -5
        keep[e * page:(e + 1) * page] = False
    tree = random_tree(nodes, np.random.default_rng(3))
    q, t = randn((1, nodes, hq, 64), BF, 4), i32(table.tolist())
    ws = bd.alloc_paged_tree_workspace(q, cache, t)
    for _ in range(2):                                # stale stages of the first hold values
        o, lse = bd.paged_tree_attn(q, cache, t, i32([n]), i32([tree]), ws, with_lse=True)
        assert bd.read_device_status(ws) == bd.DEV_BAD_INDEX
        k, v = rows_of(cache, np.where((table < 0) | (table > 10 ** 5), 0, table), 0, n)
        seen, _ = tree_mask(n - nodes, tree)
        ro, rl, ob, lb = attend_masked(f64(q[0]), k, v, BF, seen & keep[None])
        check(f64(lse[0]), rl, lb, "lse")
        check(f64(o[0]), ro, ob, "O")


def test_long_cache_past_32_bit_offsets():
    """A pool of more than 2^31 elements: the tree's pages lie at its far end."""
    page, hkv, d = 256, 8, 128
    pages = (1 << 31) // (page * hkv * d) + 40
    cache = {x: torch.empty((pages, hkv, page, d), dtype=BF, device="cuda") for x in "KV"}
    for i, x in enumerate("KV"):
        cache[x][-12:] = randn((12, hkv, page, d), BF, i)
    table = np.arange(pages - 1, pages - 12, -1)[None]
    n, tree = 2700, random_tree(40, np.random.default_rng(5))
    q = randn((1, 40, 32, d), BF, 6, 2.0)
    o, lse = bd.paged_tree_attn(q, cache, i32(table.tolist()), i32([n]), i32([tree]), with_lse=True)
    k, v = (np.concatenate([f64(cache[x][int(p)]) for p in table[0]], 1)[:, :n].transpose(1, 0, 2)
            for x in "KV")
    ro, rl, ob, lb = attend_masked(f64(q[0]), k, v, BF, tree_mask(n - 40, tree)[0])
    check(f64(lse[0]), rl, lb, "lse")
    check(f64(o[0]), ro, ob, "O")

"""GPU checks of calls on pages beside the attentions that read them: as a serving
loop strings them together, captured and replayed, over windows that give back
what they leave behind."""

import numpy as np
import pytest
import torch

from dense_common import check, f64
from mask_common import attend_masked, window_mask
from wavelet_guided_sparse_gb300 import binding as bd

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
MAX = 2 ** 31 - 1


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def randn(shape, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def random_tree(n, rng):
    return [-1] + [int(rng.integers(-1, i)) if rng.random() < 0.5 else i - 1 for i in range(1, n)]


class Serving:
    """Two sequences that draft and keep, and the child of one, over shared pages:
    every tensor of a step is there before it, so that it can be captured."""
    SEQS, NODES, PAGE, WIDTH, PAGES = 3, 7, 16, 40, 110
    WINDOW, SINKS = 50, 5

    def __init__(self, dtype, hq, hkv, d):
        self.freq = bd.rope_inv_freq(d)
        self.layers = [{x: randn((self.PAGES, hkv, self.PAGE, d), dtype, 10 * i + j)
                        for j, x in enumerate("KV")} for i in range(2)]
        self.pools = bd.page_pools(self.layers)
        self.table = bd.alloc_page_table(self.SEQS, self.WIDTH, "cuda")
        self.refs = bd.alloc_page_refs(self.PAGES, "cuda")
        self.ws = bd.alloc_pages_workspace(self.pools, self.table, max_forks=1,
                                           max_keep=self.NODES)
        s, n = self.SEQS, self.NODES
        self.k, self.v = torch.empty((2, 2 * n, hkv, d), dtype=dtype, device="cuda")
        self.q = torch.empty((s, n, hq, d), dtype=dtype, device="cuda")
        names = ("held", "grown", "drafted", "kept", "first", "end", "zero", "over")
        self.i = {x: torch.zeros(s, dtype=torch.int32, device="cuda") for x in names}
        self.i["over"].fill_(MAX)
        self.cu, self.pos = i32([0, n, 2 * n, 2 * n]), i32([0] * (2 * n))
        self.parents, self.lists = i32([[-1] * n] * s), i32([[0] * n] * s)
        self.count, self.nodes = i32([0] * s), i32([n, n, 0])
        self.src, self.dst = i32([0]), i32([2])
        self.tree_ws = bd.alloc_paged_tree_workspace(self.q, self.layers[0], self.table)
        self.token_ws = bd.alloc_paged_attn_workspace(self.q[:, :1].contiguous(), self.layers[0],
                                                      self.table)
        self.q1 = torch.empty((s, 1, hq, d), dtype=dtype, device="cuda")
        self.tree, self.token = torch.empty_like(self.q), torch.empty_like(self.q1)

    def fill(self, step, held):
        """New drafts and lists for the two sequences; returns what they hold then."""
        rng = np.random.default_rng(step)
        n, s = self.NODES, self.SEQS
        for x, seed in ((self.k, 1), (self.v, 2), (self.q, 3), (self.q1, 4)):
            x.copy_(randn(x.shape, x.dtype, 100 * step + seed))
        count = [int(rng.integers(1, n + 1)) for _ in range(2)]
        lists = [sorted(rng.choice(n, c, replace=False).tolist()) for c in count]
        total, kept = [h + n for h in held], [h + c for h, c in zip(held, count)]
        self.i["held"].copy_(i32(held + [0]))
        self.i["drafted"].copy_(i32(total + [0]))
        self.i["kept"].copy_(i32(kept + [kept[0]]))
        self.i["first"].copy_(i32([self.SINKS] * 2 + [0]))
        self.i["end"].copy_(i32([m - self.WINDOW for m in kept] + [MAX]))
        self.parents.copy_(i32([random_tree(n, rng) for _ in range(s)]))
        self.pos.copy_(i32([h + int(rng.integers(0, 4)) for h in held for _ in range(n)]))
        self.lists.copy_(i32([[h + r for r in x] + [0] * (n - len(x))
                              for h, x in zip(held + [0], lists + [[]])]))
        self.count.copy_(i32(count + [0]))
        return kept

    def step(self, pause=lambda: None):
        def calls():
            yield bd.paged_reserve(self.pools, self.table, self.refs, self.i["drafted"], self.ws)
            for c in self.layers:
                yield bd.paged_append(self.k, self.v, c, self.table, self.cu, self.i["held"],
                                      inv_freq=self.freq, positions=self.pos, ws=self.ws)
            yield bd.paged_tree_attn(self.q, self.layers[1], self.table, self.i["drafted"],
                                     self.parents, self.tree_ws, tree_len=self.nodes,
                                     out=self.tree)
            yield bd.paged_keep(self.pools, self.table, self.i["drafted"], self.i["held"],
                                self.lists, self.count, self.refs, self.ws)
            yield bd.paged_fork(self.pools, self.table, self.refs, self.src, self.dst,
                                self.i["kept"], ws=self.ws)
            yield bd.paged_window_attn(self.q1, self.layers[0], self.table, self.i["kept"],
                                       self.WINDOW, self.token_ws, sinks=self.SINKS,
                                       out=self.token)
            yield bd.paged_release(self.pools, self.table, self.refs, self.i["first"],
                                   self.i["end"], self.ws)
        for _ in calls():
            pause()

    def everything(self):
        return [self.table, self.refs, self.tree, self.token, *self.pools.tensors]

    def status(self):
        return [bd.read_device_status(w) for w in (self.ws, self.tree_ws, self.token_ws)]


@pytest.mark.parametrize("dtype,hq,hkv,d", [(BF, 8, 2, 128), (BF, 2, 2, 64), (F32, 4, 2, 64)])
def test_a_captured_serving_loop_is_the_same_calls_one_by_one(dtype, hq, hkv, d):
    """Kernels that follow one another at once, over tables, counts and rows that the last
    one has just written, replayed with other lengths and lists."""
    a, b = Serving(dtype, hq, hkv, d), Serving(dtype, hq, hkv, d)
    held = [90, 33]
    for x in (a, b):
        for w in (x.tree_ws, x.token_ws):
            w.zero_()
    graph = torch.cuda.CUDAGraph()
    a.fill(0, held)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        a.step()
    for step in range(12):
        a.fill(step, held)
        kept = b.fill(step, held)
        torch.cuda.synchronize()
        graph.replay()
        b.step(torch.cuda.synchronize)
        torch.cuda.synchronize()
        for x, y in zip(a.everything(), b.everything()):
            assert torch.equal(x, y), step
        held = kept
        assert a.status() == b.status() == [0, 0, 0], step


def test_captured_on_two_streams_that_meet():
    """A call launched early behind an event of another stream waits for both."""
    hkv, d, n = 2, 64, 300
    cache = {x: randn((30, hkv, 16, d), BF, i) for i, x in enumerate("KV")}
    table, lens = i32([list(range(25))]), i32([n])
    q, new = randn((1, 6, 4, d), BF, 5), randn((2, 6, hkv, d), BF, 6)
    tree = i32([[-1, 0, 0, 1, 2, 2]])
    ws = bd.alloc_paged_tree_workspace(q, cache, table)
    out, copy = torch.empty_like(q), torch.empty_like(q)
    side = torch.cuda.Stream()

    def calls():
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        with torch.cuda.stream(side):                # the last six rows, from the other stream
            bd.paged_append(new[0], new[1], cache, table, i_cu, i_len)
        copy.copy_(q)
        here.wait_stream(side)
        bd.paged_tree_attn(copy, cache, table, lens, tree, ws, out=out)

    i_cu, i_len = i32([0, 6]), i32([n - 6])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for seed in range(5):
        new.copy_(randn(new.shape, BF, 20 + seed))
        q.copy_(randn(q.shape, BF, 40 + seed))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, bd.paged_tree_attn(q, cache, table, lens, tree))
    assert bd.read_device_status(ws) == 0


def test_more_entries_than_32_bits_count():
    """Sequences that want 2^31 pages in all: those that there are go to the first ones."""
    seqs, width = 4096, 1 << 19
    cache = {x: torch.empty((60, 1, 8, 64), dtype=BF, device="cuda") for x in "KV"}
    table = bd.alloc_page_table(seqs, width, "cuda")
    refs = bd.alloc_page_refs(60, "cuda")
    refs[7] = 1
    ws = bd.alloc_pages_workspace(cache, table)
    bd.paged_reserve(cache, table, refs, i32([8 * width] * seqs), ws)
    assert bd.read_device_status(ws) == bd.DEV_NO_PAGE
    want = [p for p in range(60) if p != 7]
    assert table[0, :59].tolist() == want and (refs == 1).all()
    table[0, :59] = -1
    assert all((part == -1).all() for part in table.split(256))


def test_reserve_from_what_is_held():
    """Entries below the first new row stay as they are, the others are filled in order."""
    page, width, seqs, pages = 8, 700, 6, 3000
    cache = {x: torch.empty((pages, 1, page, 64), dtype=BF, device="cuda") for x in "KV"}
    rng = np.random.default_rng(4)
    order = rng.permutation(pages)[:2000].tolist()
    table = np.full((seqs, width), -1)
    refs = [0] * pages
    for s in range(seqs):
        for e in range(width):
            if rng.random() < 0.4:
                table[s, e] = order.pop()
                refs[table[s, e]] = 1
    start = [0, 3, 8 * 300, 8 * 300 + 1, 5600, 40]
    rows = [50, 4, 8 * 300, 8 * 600, 5600, 5598]
    got_t, got_r = i32(table.tolist()), i32(refs)
    ws = bd.alloc_pages_workspace(cache, got_t)
    bd.paged_reserve(cache, got_t, got_r, i32(rows), ws, from_rows=i32(start))
    for s in range(seqs):
        for e in range(start[s] // page, -(-rows[s] // page) if rows[s] > start[s] else 0):
            if table[s, e] < 0:
                table[s, e] = refs.index(0)
                refs[table[s, e]] = 1
    assert got_t.tolist() == table.tolist() and got_r.tolist() == refs
    assert bd.read_device_status(ws) == 0
    for bad in (-1, width * page + 1):
        bd.clear_device_status(ws)
        bd.paged_reserve(cache, got_t, got_r, i32([0] * seqs), ws, from_rows=i32([bad] * seqs))
        assert bd.read_device_status(ws) == bd.DEV_BAD_INDEX
    assert got_t.tolist() == table.tolist()


@pytest.mark.parametrize("dtype,new,hq,hkv,d", [(BF, 1, 8, 2, 64), (BF, 7, 4, 2, 128),
                                                (F32, 5, 2, 1, 64)])
def test_a_window_in_a_pool_of_its_own_size(dtype, new, hq, hkv, d):
    """Sequences several windows long, in pages for little more than one window each."""
    page, window, sinks, steps = 16, 100, 20, 600 // new + 1
    # A sequence's first tokens, its window with the last and the new rows, a page cut at the end.
    pool = 2 * (-(-sinks // page) + -(-(window + 2 * new - 1) // page) + 1)
    cache = {x: torch.full((pool, hkv, page, d), float("nan"), dtype=dtype, device="cuda")
             for x in "KV"}
    table, refs = bd.alloc_page_table(2, 60, "cuda"), bd.alloc_page_refs(pool, "cuda")
    ws = bd.alloc_pages_workspace(cache, table)
    held = [0, 37]
    past = [[torch.zeros((0, hkv, d), dtype=dtype, device="cuda") for _ in "KV"] for _ in held]
    first = randn((2, 37, hkv, d), dtype, 1)
    bd.paged_reserve(cache, table, refs, i32(held), ws)
    bd.paged_append(first[0], first[1], cache, table, i32([0, 0, 37]), i32([0, 0]), ws=ws)
    past[1] = [first[0], first[1]]
    qs = randn((2, new, hq, d), dtype, 2)
    ws_attn = bd.alloc_paged_attn_workspace(qs, cache, table)
    for step in range(steps):
        k, v = randn((2, 2 * new, hkv, d), dtype, 10 + step)
        lens, grown = i32(held), i32([h + new for h in held])
        bd.paged_reserve(cache, table, refs, grown, ws, from_rows=lens)
        bd.paged_append(k, v, cache, table, i32([0, new, 2 * new]), lens, ws=ws)
        o = bd.paged_window_attn(qs, cache, table, grown, window, ws_attn, sinks=sinks)
        bd.paged_release(cache, table, refs, i32([sinks] * 2), grown - new - window + 1, ws)
        for s in range(2):
            past[s] = [torch.cat((x, y[s * new:(s + 1) * new])) for x, y in zip(past[s], (k, v))]
        held = [h + new for h in held]
        if step % 40 and step + 1 < steps:
            continue
        for s, n in enumerate(held):
            seen = window_mask(n - new + np.arange(new), n, window, sinks, True)
            ro, _, ob, _ = attend_masked(f64(qs[s]), *[f64(x) for x in past[s]], dtype, seen)
            check(f64(o[s]), ro, ob, f"O of sequence {s}, step {step}")
    assert held[0] > 5 * window
    assert bd.read_device_status(ws) == 0 and bd.read_device_status(ws_attn) == 0
    assert refs.sum() == (table >= 0).sum() and refs.max() == 1


@pytest.mark.parametrize("share", [None, 0, 150, 500])
def test_a_windowed_sequence_forks_as_it_is(share):
    """What the parent has given back stays without a page in the child: no flag, no page taken,
    and the child's window is the parent's."""
    page, hkv, d, window, sinks, n = 16, 2, 64, 100, 20, 700
    cache = {x: randn((150, hkv, page, d), BF, i) for i, x in enumerate("KV")}
    table, refs = bd.alloc_page_table(3, 60, "cuda"), bd.alloc_page_refs(150, "cuda")
    ws = bd.alloc_pages_workspace(cache, table, max_forks=2)
    bd.paged_reserve(cache, table, refs, i32([n, 0, 0]), ws)
    bd.paged_release(cache, table, refs, i32([sinks, 0, 0]), i32([n - window, 0, 0]), ws)
    held = refs.sum().item()
    before = table.tolist()[0]
    rows = None if share is None else i32([share] * 2)
    bd.paged_fork(cache, table, refs, i32([0, 0]), i32([1, 2]), i32([n, 0, 0]), rows, ws)
    assert bd.read_device_status(ws) == 0
    got = table.tolist()
    assert got[0] == before
    shared = (n if share is None else share) // page
    free = iter(sorted(set(range(150)) - {p for p in before if p >= 0}))
    for child in (1, 2):
        for e, p in enumerate(before):
            assert got[child][e] == (p if p < 0 or e < shared else next(free))
    counts = [0] * 150
    for p in got[0] + got[1] + got[2]:
        if p >= 0:
            counts[p] += 1
    assert refs.tolist() == counts and sum(counts) == 3 * held
    q = randn((1, 1, 4, d), BF, 9).expand(3, 1, 4, d).contiguous()
    o = bd.paged_window_attn(q, cache, table, i32([n] * 3), window, sinks=sinks)
    assert torch.equal(o[0], o[1]) and torch.equal(o[0], o[2])


def test_a_fork_of_entries_outside_the_pool_is_flagged():
    cache = {x: randn((30, 1, 8, 64), BF, i) for i, x in enumerate("KV")}
    table, refs = bd.alloc_page_table(2, 6, "cuda"), bd.alloc_page_refs(30, "cuda")
    ws = bd.alloc_pages_workspace(cache, table, max_forks=1)
    bd.paged_reserve(cache, table, refs, i32([41, 0]), ws)
    table[0, 1] = table[0, 4] = 30
    bd.paged_fork(cache, table, refs, i32([0]), i32([1]), i32([41, 0]), i32([24]), ws)
    assert bd.read_device_status(ws) == bd.DEV_BAD_INDEX
    # Entry 1 was to be shared; 3, 4 and 5 take fresh pages, into that of 4 nothing is copied.
    assert table[1].tolist() == [0, -1, 2, 6, 7, 8]
    assert refs.tolist() == [2, 1, 2, 1, 1, 1, 1, 1, 1] + [0] * 21
    for x in cache.values():
        assert torch.equal(x[6], x[3]) and torch.equal(x[8, :, :1], x[5, :, :1])


@pytest.mark.parametrize("width", [6, 700])
def test_a_fork_into_a_child_with_pages_is_skipped(width):
    """Its references would be lost; the other forks of the call go on."""
    cache = {x: randn((60, 1, 8, 64), BF, i) for i, x in enumerate("KV")}
    table, refs = bd.alloc_page_table(5, width, "cuda"), bd.alloc_page_refs(60, "cuda")
    ws = bd.alloc_pages_workspace(cache, table, max_forks=3)
    bd.paged_reserve(cache, table, refs, i32([41, 0, 0, 0, 9]), ws)
    table[1, width - 1], refs[50] = 50, 1             # one page, behind everything
    bd.paged_fork(cache, table, refs, i32([0, 0, 0]), i32([1, 2, 4]), i32([41, 0, 0, 0, 9]),
                  i32([0, 16, 0]), ws)
    assert bd.read_device_status(ws) == bd.DEV_BAD_INDEX
    rest = [-1] * (width - 6)
    assert table.tolist() == [[0, 1, 2, 3, 4, 5] + rest, [-1] * (width - 1) + [50],
                              [0, 1, 8, 9, 10, 11] + rest, [-1] * width,
                              [6, 7] + [-1] * (width - 2)]
    assert refs.tolist() == [2, 2] + [1] * 10 + [0] * 38 + [1] + [0] * 9


@pytest.mark.parametrize("most", [20, 300])
@pytest.mark.parametrize("same", ["layer", "values"])
def test_a_pool_named_twice_is_moved_once(most, same):
    """Rows move up in place: a second stream over the same ones would read what the first has
    written."""
    page, hkv, d, n = 16, 4, 128, 900
    k, v = (randn((60, hkv, page, d), BF, i) for i in range(2))
    layers = [{"K": k, "V": v}] * 3 if same == "layer" else [{"K": k, "V": k}]
    table, refs = bd.alloc_page_table(1, 60, "cuda"), bd.alloc_page_refs(60, "cuda")
    ws = bd.alloc_pages_workspace(layers[0], table, max_keep=most)
    for seed in range(10):
        bd.paged_reserve(layers[0], table, refs, i32([n]), ws)
        rows = {x: t[table[0, :57].long()].transpose(1, 2).flatten(0, 1)[:n].clone()
                for x, t in (("K", k), ("V", v))}
        kept = sorted(np.random.default_rng(seed).choice(n, most, replace=False).tolist())
        bd.paged_keep(layers, table, i32([n]), i32([0]), i32([kept]), i32([most]), refs, ws)
        assert bd.read_device_status(ws) == 0
        for x, t in (("K", k), ("V", v))[:2 if same == "layer" else 1]:
            got = t[table[0, :-(-most // page)].long()].transpose(1, 2).flatten(0, 1)[:most]
            assert torch.equal(got, rows[x][kept])
        bd.paged_release(layers[0], table, refs, i32([0]), i32([MAX]), ws)


@pytest.mark.parametrize("width", [40, 700])
def test_entries_behind_a_childs_rows_become_minus_one(width):
    """Whatever negative number said that there was no page."""
    cache = {x: randn((60, 1, 8, 64), BF, i) for i, x in enumerate("KV")}
    table, refs = bd.alloc_page_table(4, width, "cuda"), bd.alloc_page_refs(60, "cuda")
    ws = bd.alloc_pages_workspace(cache, table, max_forks=2)
    bd.paged_reserve(cache, table, refs, i32([41, 0, 0, 0]), ws)
    table[2], table[3, 1::3] = -9, -2
    bd.paged_fork(cache, table, refs, i32([0, 0]), i32([2, 3]), i32([41, 0, 0, 0]), i32([41, 16]), ws)
    assert bd.read_device_status(ws) == 0
    rest = [-1] * (width - 6)
    assert table[2:].tolist() == [[0, 1, 2, 3, 4, 6] + rest, [0, 1, 7, 8, 9, 10] + rest]

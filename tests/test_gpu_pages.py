"""GPU checks of the pages of a paged cache (reserve, fork, keep, release)
against the rules entry by entry and row by row, bit for bit."""

import numpy as np
import pytest
import torch

from wavelet_guided_sparse_gb300 import binding as bd

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
MAX = 2 ** 31 - 1


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Model:
    """A pool of `layers` layers on the GPU and the same on the host."""

    def __init__(self, pages, width, seqs, page, hkv=2, d=64, dtype=BF, layers=2, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        word = torch.int16 if dtype == BF else torch.int32
        # Any bit pattern, NaN and infinities among them, moves as it is.
        shape = (layers, 2, pages, hkv, page, d)
        self.bits = torch.randint(-2 ** 15, 2 ** 15, shape, generator=g, device="cuda",
                                  dtype=torch.int32).to(word)
        self.caches = [{"K": x[0], "V": x[1]} for x in self.bits.view(dtype)]
        self.host = self.bits.cpu().numpy()
        self.page, self.pages, self.width = page, pages, width
        self.table = bd.alloc_page_table(seqs, width, "cuda")
        self.refs = bd.alloc_page_refs(pages, "cuda")
        self.t = self.table.tolist()
        self.r = [0] * pages
        self.ws = bd.alloc_pages_workspace(self.caches[0], self.table, max_forks=seqs,
                                           max_keep=width * page)
        self.flags = 0

    def need(self, n):
        return -(-n // self.page)

    def take(self):
        if 0 not in self.r:
            self.flags |= bd.DEV_NO_PAGE
            return -1
        p = self.r.index(0)
        self.r[p] = 1
        return p

    def reserve(self, rows, **kw):
        bd.paged_reserve(self.caches[0], self.table, self.refs, i32(rows), self.ws, **kw)
        for s, n in enumerate(rows):
            if not 0 <= n <= self.width * self.page:
                self.flags |= bd.DEV_BAD_INDEX
            for e in range(self.need(min(max(n, 0), self.width * self.page))):
                if self.t[s][e] < 0:
                    self.t[s][e] = self.take()

    def fork(self, src, dst, lens, share=None):
        bd.paged_fork(self.caches, self.table, self.refs, i32(src), i32(dst), i32(lens),
                      None if share is None else i32(share), self.ws)
        fresh = []
        for i, (a, b) in enumerate(zip(src, dst)):
            if not (0 <= a < len(self.t) and 0 <= b < len(self.t)):
                self.flags |= bd.DEV_BAD_INDEX
                continue
            if b in src or dst.count(b) > 1:
                self.flags |= bd.DEV_DUP_INDEX
                continue
            full = min(lens[a] if share is None else share[i], lens[a]) // self.page
            self.t[b] = [-1] * self.width
            for e in range(full):
                self.t[b][e] = self.t[a][e]
                self.r[self.t[a][e]] += 1
            fresh += [(a, b, e) for e in range(full, self.need(lens[a]))]
        for a, b, e in fresh:
            p = self.t[b][e] = self.take()
            if p >= 0:
                n = min(self.page, lens[a] - e * self.page)
                self.host[:, :, p, :, :n] = self.host[:, :, self.t[a][e], :, :n]

    def drop(self, s, first, end):
        for e in range(self.width):
            if e * self.page >= first and (e + 1) * self.page <= end and self.t[s][e] >= 0:
                self.r[self.t[s][e]] -= 1
                self.t[s][e] = -1

    def keep(self, lens, start, lists=None, refs=True, skip=(), most=None):
        call = {}
        if lists is not None:
            most = most or max(1, max(len(x) for x in lists))
            call = dict(keep=i32([x + [0] * (most - len(x)) for x in lists]),
                        n_keep=i32([len(x) for x in lists]))
        bd.paged_keep(bd.page_pools(self.caches), self.table, i32(lens), i32(start), ws=self.ws,
                      refs=self.refs if refs else None, **call)
        before = self.host.copy()
        for s in range(len(self.t)):
            if s in skip:
                continue
            rows = [] if lists is None else lists[s]
            for i, old in enumerate(rows):
                new = start[s] + i
                self.host[:, :, self.t[s][new // self.page], :, new % self.page] = \
                    before[:, :, self.t[s][old // self.page], :, old % self.page]
            if refs:
                self.drop(s, start[s] + len(rows), MAX)

    def release(self, first, end):
        bd.paged_release(self.caches[0], self.table, self.refs, i32(first), i32(end), self.ws)
        for s in range(len(self.t)):
            self.drop(s, max(first[s], 0), end[s])

    def check(self, flags=None):
        assert self.table.tolist() == self.t
        assert self.refs.tolist() == self.r
        np.testing.assert_array_equal(self.bits.cpu().numpy(), self.host)
        assert bd.read_device_status(self.ws) == (self.flags if flags is None else flags)


@pytest.mark.parametrize("page,d,dtype,layers,hkv", [
    (16, 128, BF, 3, 2), (8, 64, BF, 1, 1), (64, 64, F32, 2, 3), (256, 128, F32, 1, 1),
    (32, 128, BF, 2, 5)])
def test_a_life_of_pages(page, d, dtype, layers, hkv):
    """Sequences grow, fork, keep rows, fork again, and end."""
    m = Model(90, 12, 6, page, hkv, d, dtype, layers, seed=page)
    top = 12 * page
    m.reserve([0, 1, page, 3 * page + 5, top, 0])
    m.check()
    lens = [0, 1, page, 3 * page + 5, top, 0]
    m.fork([3, 4], [0, 5], lens)                    # shared; a parent whose last page is full
    lens[0], lens[5] = lens[3], lens[4]
    m.check()
    m.reserve([3 * page + 9, 9, page + 1, 0, top, top])
    m.check()
    m.release([0, 0, 0, 0, 0, page + 1], [0, MAX, 0, MAX, 0, 5 * page - 1])
    m.check()                                        # shared pages stay with the others
    m.fork([4, 2], [3, 1], lens, share=[2 * page + 3, 0])
    lens[3], lens[1] = lens[4], lens[2]
    m.check()
    rng = np.random.default_rng(page)
    rows = sorted(rng.choice(np.arange(2 * page + 1, top), 2 * page + 3, replace=False).tolist())
    m.keep([0, 0, page, top, 0, 0], [0, 0, 0, 2 * page, 0, 0],
           [[], [], list(range(0, page, 3)), rows, [], []])
    m.check()
    m.keep([lens[s] if s == 5 else 0 for s in range(6)], [0] * 6)   # nothing but frees
    m.check()
    assert m.refs.sum().item() == sum(p >= 0 for row in m.t for p in row)


@pytest.mark.parametrize("most,n", [(1, 1), (7, 7), (32, 32), (33, 33), (129, 129), (700, 641)])
@pytest.mark.parametrize("d,dtype", [(64, BF), (128, BF), (128, F32)])
def test_rows_that_move_over_their_own_places(most, n, d, dtype):
    """Dense lists, whose destinations are other kept rows' old places."""
    m = Model(200, 60, 3, 16, 3, d, dtype, 2, seed=most)
    lens = [900, 960, 700]
    m.reserve(lens)
    rng = np.random.default_rng(n)
    lists = [list(range(3, 3 + n)), sorted(rng.choice(960, n, replace=False).tolist()),
             [9 + i for i in range(min(n, 5))] + [15 + i for i in range(n - min(n, 5))]]
    m.keep(lens, [0, 0, 9], lists, most=most)         # the third one's first rows stay
    m.check()


def test_no_rows_of_other_sequences_change_without_refs():
    m = Model(40, 8, 2, 32, 2, 128, F32, 1, seed=3)
    m.reserve([200, 150])
    m.keep([200, 150], [10, 0], [[12, 40, 41, 199], []], refs=False)
    m.check()


def test_large_pools_take_the_lowest_pages_in_order():
    pages = 40000                                     # a cluster counts
    m = Model(pages, 300, 5, 8, 1, 64, BF, 1, seed=1)
    held = np.random.default_rng(2).permutation(pages)[: pages - 900].tolist()
    for p in held:
        m.r[p] = 1
    m.refs.copy_(i32(m.r))
    m.reserve([2000, 3, 0, 1600, 0])
    m.check()
    m.fork([0, 3], [2, 4], [2000, 3, 0, 1600, 0], share=[8 * 100, 0])
    m.check()


@pytest.mark.parametrize("pages", [12000, 20000])
def test_more_pages_at_once_than_one_list_holds(pages):
    m = Model(pages, 1500, 5, 8, 1, 64, BF, 1, seed=pages)
    held = np.random.default_rng(5).permutation(pages)[:1500].tolist()
    for p in held:
        m.r[p] = 1
    m.refs.copy_(i32(m.r))
    m.reserve([12000, 9001, 8, 11999, 0])             # 4127 pages: one CTA, a cluster
    m.check()
    m.release([8, 0, 0, 16, 0], [11992, 0, MAX, 800, 0])
    m.reserve([12000, 10000, 0, 0, 0])
    m.check()


def test_captured_calls_on_a_large_pool():
    m = Model(40000, 40, 3, 8, 1, 64, BF, 1, seed=14)
    held = np.random.default_rng(3).permutation(40000)[:39000].tolist()
    for p in held:
        m.r[p] = 1
    m.refs.copy_(i32(m.r))
    rows, first, end = i32([300, 0, 77]), i32([0] * 3), i32([MAX] * 3)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        bd.paged_reserve(m.caches[0], m.table, m.refs, rows, m.ws)
        taken = m.table.clone()
        bd.paged_release(m.caches[0], m.table, m.refs, first, end, m.ws)
    free = [p for p in range(40000) if m.r[p] == 0]
    want = [free[:38] + [-1] * 2, [-1] * 40, free[38:48] + [-1] * 30]
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert taken.tolist() == want
        m.check()


def test_pools_past_32_bit_offsets():
    """More than 2^31 elements a pool: rows at its far end are copied and moved."""
    page, hkv, d = 256, 8, 128
    pages = (1 << 31) // (page * hkv * d) + 40
    cache = {x: torch.empty((pages, hkv, page, d), dtype=BF, device="cuda") for x in "KV"}
    g = torch.Generator(device="cuda").manual_seed(1)
    for x in cache.values():
        x[-12:].normal_(generator=g)
    refs = torch.ones(pages, dtype=torch.int32, device="cuda")
    table = bd.alloc_page_table(2, 6, "cuda")
    refs[-12:] = 0
    ws = bd.alloc_pages_workspace(cache, table, max_forks=1, max_keep=600)
    bd.paged_reserve(cache, table, refs, i32([1300, 0]), ws)
    assert table[0].tolist() == list(range(pages - 12, pages - 6))
    bd.paged_fork(cache, table, refs, i32([0]), i32([1]), i32([1300, 0]), i32([0]), ws)
    assert table[1].tolist() == list(range(pages - 6, pages))
    rows = {x: [t[table[s].long()].transpose(1, 2).flatten(0, 1)[:1300].clone() for s in (0, 1)]
            for x, t in cache.items()}
    for x in rows.values():
        assert torch.equal(x[0], x[1])
    kept = sorted(np.random.default_rng(2).choice(1300, 600, replace=False).tolist())
    bd.paged_keep(cache, table, i32([1300, 1300]), i32([0, 1300]), i32([kept, [0] * 600]),
                  i32([600, 0]), refs, ws)
    assert bd.read_device_status(ws) == 0 and (refs[-12:] == 0).sum() == 3
    for x, t in cache.items():
        got = t[table[0, :3].long()].transpose(1, 2).flatten(0, 1)[:600]
        assert torch.equal(got, rows[x][0][kept])
        assert torch.equal(t[table[1].long()].transpose(1, 2).flatten(0, 1)[:1300], rows[x][1])


def test_too_few_pages():
    m = Model(10, 6, 3, 8, seed=4)
    m.reserve([40, 48, 0])                            # 5 + 6 of 10
    m.check(bd.DEV_NO_PAGE)
    m = Model(10, 6, 3, 8, seed=5)
    m.reserve([40, 0, 0])
    m.fork([0], [1], [40, 0, 0], share=[0])           # the other five
    m.check(0)
    m.fork([0], [2], [39, 0, 0])                      # four shared, none for the last one
    m.check(bd.DEV_NO_PAGE)


def test_unsound_forks_are_skipped():
    m = Model(60, 4, 8, 16, seed=6)
    lens = [30, 64, 20, 0, 0, 0, 0, 0]
    m.reserve(lens)
    m.fork([0, 1, 9, 2, 2, 0, -1], [3, 4, 5, 1, 5, 5, 6], lens)
    assert m.flags == bd.DEV_BAD_INDEX | bd.DEV_DUP_INDEX
    m.check()


def test_lists_that_break_the_rules_leave_their_sequence_alone():
    m = Model(60, 6, 9, 16, seed=7)
    lens = [90] * 9
    m.reserve(lens)
    lists = [[5, 9, 90], [9, 8], [7, 7], [3], [20, 30], [40, 41], [1], [60], [2, 50]]
    start = [0, 0, 0, 4, 10, 40, 0, 91, 0]
    lens[6] = 97                                     # behind the table
    m.table[8, 3] = m.t[8][3] = 60                   # row 50 has no page
    m.keep(lens, start, lists, skip=(0, 1, 2, 3, 6, 7, 8))
    m.check(bd.DEV_BAD_INDEX)


def test_lists_longer_than_what_lies_behind_their_start():
    m = Model(60, 6, 4, 16, seed=12)
    lens = [96, 96, 90, 96]
    m.reserve(lens)
    lists = [[50, 51] * 40, [95] * 96, list(range(80, 90)) * 8, list(range(96))]
    m.keep(lens, [50, 90, 80, 0], lists, skip=(0, 1, 2))
    m.check(bd.DEV_BAD_INDEX)


def test_shared_pages_are_not_written():
    m = Model(60, 6, 3, 16, seed=8)
    m.reserve([90, 0, 0])
    m.fork([0], [1], [90, 0, 0])
    m.check()
    # Rows 3.. would move into a shared page; the child's own last page may take rows.
    m.keep([90, 90, 0], [0, 80, 0], [[3, 4], [83, 89], []], skip=(0,))
    m.check(bd.DEV_SHARED_PAGE)


def test_released_twice_is_flagged():
    m = Model(8, 3, 2, 16, seed=9)
    m.reserve([40, 0])
    m.table[1] = m.table[0]                          # three entries nobody counted
    bd.paged_release(m.caches[0], m.table, m.refs, i32([0, 0]), i32([MAX, MAX]), m.ws)
    assert (m.table == -1).all() and (m.refs == 0).all()
    assert bd.read_device_status(m.ws) == bd.DEV_BAD_INDEX


def test_captured_calls_follow_the_tables():
    m = Model(64, 6, 4, 16, 2, 64, BF, 2, seed=10)
    m.reserve([90, 33, 0, 0])
    lens, rows = i32([90, 33, 0, 0]), i32([90, 60, 0, 0])
    src, dst, first = i32([0]), i32([2]), i32([0] * 4)
    end, start = i32([0, 0, MAX, 0]), i32([80, 30, 0, 0])
    keep, count = i32([[84, 89], [31, 32], [0, 0], [0, 0]]), i32([2, 2, 0, 0])
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    pools = bd.page_pools(m.caches)
    with torch.cuda.graph(graph):
        bd.paged_reserve(pools, m.table, m.refs, rows, m.ws)
        bd.paged_fork(pools, m.table, m.refs, src, dst, lens, ws=m.ws)
        bd.paged_release(pools, m.table, m.refs, first, end, m.ws)
        bd.paged_keep(pools, m.table, lens, start, keep, count, m.refs, m.ws)
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        for s, n in enumerate([90, 60, 0, 0]):
            for e in range(m.need(n)):
                if m.t[s][e] < 0:
                    m.t[s][e] = m.take()
        p = m.take()                                  # the fork's partial page
        a, n = m.t[0][5], 90 - 80
        m.host[:, :, p, :, :n] = m.host[:, :, a, :, :n]
        m.r[p] = 0
        before = m.host.copy()
        for s, at, old in ((0, 80, 84), (0, 81, 89), (1, 30, 31), (1, 31, 32)):
            m.host[:, :, m.t[s][at // 16], :, at % 16] = \
                before[:, :, m.t[s][old // 16], :, old % 16]
        m.drop(0, 82, MAX)
        m.drop(1, 32, MAX)
        m.check()


def test_on_another_stream():
    m = Model(64, 6, 4, 16, seed=11)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    m.reserve([90, 33, 0, 0], stream=side)
    side.synchronize()
    m.check()
    with pytest.raises(ValueError):
        bd.paged_keep(m.caches, m.table, i32([0] * 4), i32([0] * 4), i32([0] * 4), i32([0] * 4),
                      m.refs, m.ws)                  # keep is not [n_seqs, max_keep]
    with pytest.raises(bd.WfError):
        bd.paged_reserve(m.caches[0], m.table, m.refs, i32([0] * 4), m.ws[:256])

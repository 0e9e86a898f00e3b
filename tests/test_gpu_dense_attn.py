"""GPU checks of the paged append, the paged attention and the packed-prompt
attention against 64-bit references, through the public entry points.  Rows no
result may depend on hold NaN or infinities."""

import math

import numpy as np
import pytest
import torch

from dense_common import attend, check, f64, half_step, rotate, rotation_bound
from wavelet_guided_sparse_gb300 import binding as bd

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def randn(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def offsets(lens):
    return i32([0] + list(np.cumsum(lens)))


def make_table(lens, page, seed, spare=2, width=None):
    """Shuffled pages per sequence, bad entries behind the used ones."""
    need = [-(-n // page) for n in lens]
    order = np.random.default_rng(seed).permutation(sum(need) + spare)
    width = width or max(max(need), 1)
    table = np.full((len(lens), width), -7, np.int64)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    return i32(table.tolist()), sum(need) + spare


def slope_list(hq):
    return torch.tensor([2.0 ** (-8 * (h + 1) / hq) for h in range(hq)], device="cuda")


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("dtype,d,hq,hkv,page,new,before,rotary,inter,keep,extra", [
    (BF, 128, 32, 8, 16, [1, 1, 1], [0, 17, 8191], 128, False, False, 0),
    (BF, 128, 4, 4, 64, [130, 0, 1, 77], [5, 3, 63, 64], 128, True, True, 3),
    (BF, 64, 6, 2, 8, [33], [131000], 32, False, True, 0),
    (BF, 128, 0, 1, 256, [300, 5], [0, 1], 16, True, False, 2),
    (F32, 64, 2, 2, 32, [100, 29], [1000000, 7], 64, False, True, 1),
    (F32, 128, 3, 1, 128, [9], [250], 48, True, False, 0),
    (F32, 64, 1, 1, 8, [4], [0], 0, False, True, 0),
    (BF, 128, 8, 8, 32, [3000], [0], 128, False, True, 0),   # several lines a thread
])
def test_append(dtype, d, hq, hkv, page, new, before, rotary, inter, keep, extra):
    t = sum(new) + extra
    fused = randn((t, hq + 2 * hkv, d), dtype, 3)     # one projection's slices: strided rows
    q = fused[:, :hq] if hq else None
    k, v = fused[:, hq:hq + hkv], fused[:, hq + hkv:]
    # Positions past a million rows need a long table: offset it to the rows used.
    shift = [b // page * page if b > 100000 else 0 for b in before]
    pos_over = None
    if any(shift):
        pos_over = i32([b + i for b, n in zip(before, new) for i in range(n)] + [0] * extra)
        before_dev = [b - s for b, s in zip(before, shift)]
    else:
        before_dev = before
    table, pages = make_table([b + n for b, n in zip(before_dev, new)], page, 5)
    cache = bd.alloc_paged_cache(pages, hkv, page, d, dtype, "cuda")
    for x in cache.values():
        x.fill_(0.25)
    out = {"Q": torch.full((t, hq, d), 7.0, dtype=dtype, device="cuda")} if hq else {}
    if keep:
        out["K"] = torch.full((t, hkv, d), 7.0, dtype=dtype, device="cuda")
    ws = bd.alloc_status_workspace("cuda")
    freq = bd.rope_inv_freq(rotary) if rotary else None
    res = bd.paged_append(k, v, cache, table, offsets(new), i32(before_dev), q=q, inv_freq=freq,
                          interleaved=inter, positions=pos_over, keep_keys=keep, out=out, ws=ws)
    assert bd.read_device_status(ws) == 0
    pos = np.concatenate([np.arange(b, b + n) for b, n in zip(before, new)])
    cpos = np.concatenate([np.arange(b, b + n) for b, n in zip(before_dev, new)])
    live = sum(new)
    fr = [] if freq is None else list(freq)
    kx = f64(k)[:live]
    kr = rotate(kx, pos, fr, inter)
    kb = rotation_bound(kx, rotary, inter, kr, dtype)
    kb[..., rotary:] = 0
    ref_k, ref_v = f64(cache["K"]) * 0 + 0.25, f64(cache["V"]) * 0 + 0.25
    bound = np.zeros_like(ref_k)
    tab = table.cpu().numpy()
    seq = np.repeat(np.arange(len(new)), new)
    for i in range(live):
        pg, r = tab[seq[i], cpos[i] // page], cpos[i] % page
        ref_k[pg, :, r], ref_v[pg, :, r], bound[pg, :, r] = kr[i], f64(v[i]), kb[i]
    check(f64(cache["K"]), ref_k, bound, "key pages")
    np.testing.assert_array_equal(f64(cache["V"]), ref_v)
    if hq:
        qx = f64(q)[:live]
        qr = rotate(qx, pos, fr, inter)
        qb = rotation_bound(qx, rotary, inter, qr, dtype)
        qb[..., rotary:] = 0
        check(f64(res["Q"])[:live], qr, qb, "queries")
        assert (res["Q"][live:] == 7).all()           # rows behind the last sequence
    if keep:
        check(f64(res["K"])[:live], kr, kb, "kept keys")
        assert (res["K"][live:] == 7).all()


def test_append_in_place_queries_and_many_sequences():
    n, hkv, d, page = 1500, 2, 64, 8
    new = [1 if i % 3 else 2 for i in range(n)]
    t = sum(new)
    q, k, v = (randn((t, hkv, d), BF, s) for s in (1, 2, 3))
    table, pages = make_table([5 + m for m in new], page, 0)
    cache = bd.alloc_paged_cache(pages, hkv, page, d, BF, "cuda")
    freq = bd.rope_inv_freq(64, 500000.0)
    q0 = f64(q)
    bd.paged_append(k, v, cache, table, offsets(new), i32([5] * n), q=q, inv_freq=freq,
                    out={"Q": q})
    pos = np.concatenate([5 + np.arange(m) for m in new])
    ref = rotate(q0, pos, list(freq), False)
    check(f64(q), ref, rotation_bound(q0, 64, False, ref, BF), "queries in place")


def test_append_flags_positions_without_a_page():
    page, d = 8, 64
    k, v = randn((12, 1, d), BF, 1), randn((12, 1, d), BF, 2)
    table = i32([[0, 99], [1, -1]])         # 99 and -1: outside the pool of 3
    cache = {n: torch.zeros((3, 1, page, d), dtype=BF, device="cuda") for n in ("K", "V")}
    ws = bd.alloc_status_workspace("cuda")
    # Sequence 0: rows 4..9 (page 0, then the bad 99); sequence 1: rows 14.. (bad, then
    # behind the table).
    bd.paged_append(k, v, cache, table, i32([0, 6, 12]), i32([4, 14]), ws=ws)
    assert bd.read_device_status(ws) == bd.DEV_BAD_INDEX
    ref = torch.zeros_like(cache["K"])
    ref[0, 0, 4:8] = k[:4, 0]
    assert torch.equal(cache["K"], ref)


# ------------------------------------------------------------------ paged attention
def run_paged(dtype, d, hq, hkv, page, lens, new, causal, prefix, cap, bias, seed=0, scale=None):
    s = len(lens)
    table, pages = make_table(lens, page, seed)
    cache = {"K": randn((pages, hkv, page, d), dtype, seed + 1),
             "V": randn((pages, hkv, page, d), dtype, seed + 2)}
    q = randn((s, new, hq, d), dtype, seed + 3, 2.0)
    # Rows behind the lengths (and pages nobody has) hold what must not matter.
    tab = table.cpu().numpy()
    live = torch.zeros((pages, page), dtype=torch.bool)
    for i, n in enumerate(lens):
        for j in range(n):
            live[tab[i, j // page], j % page] = True
    dead = ~live.cuda()
    for x, bad in ((cache["K"], math.nan), (cache["V"], math.inf)):
        x.masked_fill_(dead[:, None, :, None], bad)
    pre = None if prefix is None else i32(prefix)
    slopes = slope_list(hq) if bias else None
    ws = bd.alloc_paged_attn_workspace(q, cache, table)
    o, lse = bd.paged_attn(q, cache, table, i32(lens), ws, causal=causal, prefix=pre, softcap=cap,
                           slopes=slopes, scale=scale, with_lse=True)
    assert bd.read_device_status(ws) == 0
    kc, vc = f64(cache["K"]), f64(cache["V"])
    for i, n in enumerate(lens):
        kk = np.concatenate([kc[p] for p in tab[i, :-(-n // page)]], 1)[:, :n] if n else \
            np.zeros((hkv, 0, d))
        vv = np.concatenate([vc[p] for p in tab[i, :-(-n // page)]], 1)[:, :n] if n else \
            np.zeros((hkv, 0, d))
        ro, rl, ob, lb = attend(f64(q[i]), kk.transpose(1, 0, 2), vv.transpose(1, 0, 2), dtype,
                                causal, 0 if prefix is None else prefix[i], cap,
                                None if slopes is None else slopes.cpu().numpy(), scale)
        check(f64(lse[i]), rl, lb, f"lse of sequence {i}")
        check(f64(o[i]), ro, ob, f"O of sequence {i}")
    return o, lse, (q, cache, table, i32(lens), ws)


PAGED = [
    # dtype, d, hq, hkv, page, lens, new, causal, prefix, cap, bias
    (BF, 128, 32, 8, 16, [1], 1, True, None, 0.0, False),
    (BF, 128, 32, 8, 16, [1, 17, 64, 65, 0, 1000], 1, True, None, 0.0, False),
    (BF, 128, 4, 4, 64, [63, 129, 300], 1, False, None, 20.0, True),
    (BF, 64, 12, 4, 8, [5, 200, 31], 5, True, [0, 150, 31], 0.0, True),
    (BF, 128, 8, 1, 32, [777], 3, True, None, 50.0, False),          # 24 rows a block
    (BF, 128, 2, 2, 256, [64, 70, 4097], 64, True, None, 0.0, False),
    (BF, 64, 6, 2, 16, [500, 90], 32, False, None, 0.0, False),      # 96 rows: two blocks
    (BF, 128, 16, 1, 16, [260], 1, True, None, 0.0, False),
    (BF, 128, 40, 1, 128, [513], 1, True, None, 0.0, False),         # 40 rows
    (BF, 64, 1, 1, 8, [3, 2], 8, True, None, 0.0, False),            # rows before any key
    (BF, 128, 8, 2, 64, [200, 64, 33, 0], 64, True, [0, 64, 7, 0], 30.0, True),  # 4 blocks
    (F32, 64, 2, 2, 32, [1056], 32, False, None, 0.0, False),
    (F32, 128, 4, 1, 16, [1, 0, 333], 1, True, None, 30.0, True),
    (F32, 128, 8, 2, 8, [500, 77, 0, 6], 5, True, None, 0.0, False),         # 20 rows, 8 boxes
    (F32, 128, 4, 1, 8, [333, 20], 16, True, [9, 20], 25.0, True),           # 64 rows
    (F32, 128, 4, 4, 256, [1000, 1], 20, False, None, 0.0, False),
    (F32, 64, 9, 3, 8, [100, 41], 4, True, [60, 0], 0.0, False),
    (F32, 128, 2, 2, 64, [3, 130], 7, True, None, 0.0, True),
]


@pytest.mark.parametrize("case", PAGED)
def test_paged(case):
    run_paged(*case)


def test_paged_long_splits_and_is_deterministic():
    o, lse, args = run_paged(BF, 128, 8, 2, 64, [9000, 30001], 1, True, None, 0.0, False)
    for _ in range(3):
        o2, lse2 = bd.paged_attn(*args, with_lse=True)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_paged_many_short_sequences():
    rng = np.random.default_rng(3)
    run_paged(BF, 64, 2, 1, 16, rng.integers(0, 90, 700).tolist(), 1, True, None, 0.0, False)


def test_paged_the_most_sequences():
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 40, 4096).tolist()
    run_paged(BF, 64, 1, 1, 32, lens, 1, True, None, 0.0, False)


def test_paged_large_scores_and_scale():
    # Scores of some hundreds: one key carries the row; nothing overflows.
    run_paged(BF, 128, 4, 2, 16, [70, 300], 2, True, None, 0.0, False, scale=4.0)


def test_paged_sequences_share_pages():
    # A common beginning: the same pages in three tables, one page twice in one.
    page, d, hkv = 16, 128, 2
    cache = {n: randn((6, hkv, page, d), BF, s) for s, n in enumerate(("K", "V"))}
    table = [[4, 0, 1], [4, 0, 2], [4, 4, 0]]
    lens = [48, 37, 40]
    q = randn((3, 1, 8, d), BF, 5, 2.0)
    o = bd.paged_attn(q, cache, i32(table), i32(lens))
    for i, n in enumerate(lens):
        kk, vv = (f64(cache[x])[table[i]].transpose(0, 2, 1, 3).reshape(-1, hkv, d)[:n]
                  for x in ("K", "V"))
        ro, _, ob, _ = attend(f64(q[i]), kk, vv, BF, True)
        check(f64(o[i]), ro, ob, f"O of sequence {i}")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_append_and_attention_behind_the_first_2_to_31_elements(dtype):
    # The pages in use lie past 2^31 elements of the cache.
    page, d, hkv, hq, lens = 256, 128, 8, 16, [300, 70]
    pages = 2 ** 31 // (page * d * hkv) + 8
    cache = bd.alloc_paged_cache(pages, hkv, page, d, dtype, "cuda")
    table = i32([[pages - 1, pages - 5], [pages - 3, 0]])
    k, v = (randn((sum(lens), hkv, d), dtype, s) for s in (1, 2))
    bd.paged_append(k, v, cache, table, offsets(lens), i32([0, 0]))
    assert torch.equal(cache["K"][pages - 5, :, :44], k[256:300].transpose(0, 1))
    q = randn((2, 1, hq, d), dtype, 3, 2.0)
    o = bd.paged_attn(q, cache, table, i32(lens))
    at = 0
    for i, n in enumerate(lens):
        ro, _, ob, _ = attend(f64(q[i]), f64(k[at:at + n]), f64(v[at:at + n]), dtype, True)
        check(f64(o[i]), ro, ob, f"O of sequence {i}")
        at += n


def test_paged_bad_pages_and_lengths_are_flagged():
    page, d, hkv = 16, 128, 1
    cache = {"K": randn((4, hkv, page, d), BF, 1), "V": randn((4, hkv, page, d), BF, 2)}
    q = randn((2, 1, 2, d), BF, 3)
    table = i32([[2, 77, 3], [0, 1, 3]])
    ws = bd.alloc_paged_attn_workspace(q, cache, table)
    o, lse = bd.paged_attn(q, cache, table, i32([40, 32]), ws, causal=False, with_lse=True)
    assert bd.read_device_status(ws) == bd.DEV_BAD_INDEX
    # The bad page's rows do not count: sequence 0 is page 2 and 8 rows of page 3.
    good = torch.cat([cache["K"][2, 0], cache["K"][3, 0, :8]])[:, None]
    goodv = torch.cat([cache["V"][2, 0], cache["V"][3, 0, :8]])[:, None]
    ro, rl, ob, lb = attend(f64(q[0]), f64(good), f64(goodv), BF, False)
    check(f64(o[0]), ro, ob, "O past a bad page")
    check(f64(lse[0]), rl, lb, "lse past a bad page")
    bd.clear_device_status(ws)
    o2 = bd.paged_attn(q, cache, i32([[2, 1, 3], [0, 1, 3]]), i32([4000, -3]), ws, causal=False)
    assert bd.read_device_status(ws) == bd.DEV_BAD_INDEX
    full = torch.cat([cache["K"][2, 0], cache["K"][1, 0], cache["K"][3, 0]])[:, None]
    fullv = torch.cat([cache["V"][2, 0], cache["V"][1, 0], cache["V"][3, 0]])[:, None]
    ro, _, ob, _ = attend(f64(q[0]), f64(full), f64(fullv), BF, False)
    check(f64(o2[0]), ro, ob, "O of a clamped length")
    assert (o2[1] == 0).all()


# ------------------------------------------------------------------ packed prompts
def run_prefill(dtype, d, hq, hkv, nq, nk, causal, prefix, cap, bias, extra=0, seed=0):
    tq, tk = sum(nq), sum(nk)
    fused = randn((tq + extra, hq, d), dtype, seed + 1, 2.0)
    kv = randn((tk + extra, 2 * hkv, d), dtype, seed + 2)
    kv[tk:] = math.nan
    k, v = kv[:, :hkv], kv[:, hkv:]
    pre = None if prefix is None else i32(prefix)
    slopes = slope_list(hq) if bias else None
    out = torch.full((tq + extra, hq, d), 7.0, dtype=dtype, device="cuda")
    ws = bd.alloc_status_workspace("cuda")
    o, lse = bd.prefill_attn(fused, k, v, offsets(nq), None if nq == nk else offsets(nk),
                             causal=causal, prefix=pre, softcap=cap, slopes=slopes, out=out,
                             with_lse=True, ws=ws)
    assert bd.read_device_status(ws) == 0
    aq = ak = 0
    for s, (a, b) in enumerate(zip(nq, nk)):
        ro, rl, ob, lb = attend(f64(fused[aq:aq + a]), f64(k[ak:ak + b]), f64(v[ak:ak + b]), dtype,
                                causal, 0 if prefix is None else prefix[s], cap,
                                None if slopes is None else slopes.cpu().numpy())
        check(f64(lse[aq:aq + a]), rl, lb, f"lse of sequence {s}")
        check(f64(o[aq:aq + a]), ro, ob, f"O of sequence {s}")
        aq, ak = aq + a, ak + b
    assert (o[tq:] == 7).all()
    return fused, k, v, o, lse


PREFILL = [
    # dtype, d, hq, hkv, n_q, n_k, causal, prefix, cap, bias, extra
    (BF, 128, 2, 2, [1], [1], True, None, 0.0, False, 0),
    (BF, 128, 4, 4, [128], [128], False, None, 0.0, False, 0),
    (BF, 128, 4, 2, [129], [129], True, None, 0.0, False, 5),
    (BF, 128, 8, 2, [700], [700], True, None, 0.0, False, 0),
    (BF, 128, 3, 1, [300, 17, 0, 1, 257], [300, 17, 0, 1, 257], True, [100, 17, 0, 0, 5], 0.0, False, 1),
    (BF, 128, 5, 5, [255, 40], [255, 40], False, None, 20.0, True, 0),
    (BF, 64, 4, 2, [513, 2], [513, 2], True, None, 30.0, False, 9),
    (BF, 64, 2, 1, [64, 90], [64, 90], False, None, 0.0, True, 0),
    (BF, 128, 2, 1, [5, 130, 3], [300, 20, 0], True, None, 0.0, False, 0),   # empty rows
    (BF, 128, 2, 2, [7, 3], [1000, 129], False, None, 0.0, False, 0),
    (BF, 64, 8, 8, [1100], [1100], True, [700], 50.0, True, 0),
    (F32, 64, 2, 2, [150, 1, 33], [150, 1, 33], True, [20, 0, 33], 0.0, False, 2),
    (F32, 128, 4, 2, [70], [200], True, None, 30.0, True, 0),
    (F32, 128, 3, 1, [65], [65], False, None, 0.0, False, 0),
    (F32, 64, 2, 1, [30, 4], [10, 0], True, None, 0.0, False, 0),            # empty rows
]


@pytest.mark.parametrize("case", PREFILL)
def test_prefill(case):
    run_prefill(*case)


@pytest.mark.parametrize("cap,bias,spread", [(5.0, False, 4.0), (5.0, True, 4.0), (1.0, True, 0.5),
                                             (200.0, False, 8.0)])
def test_prefill_caps_far_into_their_bend(cap, bias, spread):
    # Scores up to many times the cap, some rows small and some large at once.
    d, n, h = 128, 300, 4
    q, k, v = (randn((n, h, d), BF, s) for s in (1, 2, 3))
    q = (q.float() * torch.linspace(0.01, spread, n, device="cuda")[:, None, None]).to(BF)
    slopes = slope_list(h) if bias else None
    o, lse = bd.prefill_attn(q, k, v, offsets([n]), softcap=cap, slopes=slopes, with_lse=True)
    ro, rl, ob, lb = attend(f64(q), f64(k), f64(v), BF, True, 0, cap,
                            None if slopes is None else slopes.cpu().numpy())
    check(f64(lse), rl, lb, "lse")
    check(f64(o), ro, ob, "O")


@pytest.mark.parametrize("cap,scale,spread", [(1e7, 1.0, 2e5), (1e-7, None, 1e-8), (1e30, None, 1.0)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_caps_far_from_one(dtype, cap, scale, spread):
    # Scores about the cap's bend (or far below it) at extreme caps: there every
    # score is good to 2^-20 of itself.
    d, n, h = 128, 200, 2
    q, k, v = (randn((n, h, d), dtype, s) for s in (1, 2, 3))
    q = (q.float() * spread).to(dtype)
    o, lse = bd.prefill_attn(q, k, v, offsets([n]), softcap=cap, scale=scale, with_lse=True)
    z = np.einsum("qhd,khd->hqk", f64(q), f64(k)) * (scale or d ** -0.5)
    bend = min(cap, np.abs(z).max())
    ro, rl, ob, lb = attend(f64(q), f64(k), f64(v), dtype, True, 0, cap, scale=scale, bend=bend)
    check(f64(lse), rl, lb, "lse")
    check(f64(o), ro, ob, "O")
    table, pages = make_table([n], 16, 0)
    cache = bd.alloc_paged_cache(pages, h, 16, d, dtype, "cuda")
    bd.paged_append(k, v, cache, table, offsets([n]), i32([0]))
    o, lse = bd.paged_attn(q[None, -9:], cache, table, i32([n]), softcap=cap, scale=scale,
                           with_lse=True)
    check(f64(lse[0]), rl[-9:], lb[-9:], "lse over pages")
    check(f64(o[0]), ro[-9:], ob[-9:], "O over pages")


def test_prefill_a_multitude_of_sequences():
    # One row each: every row is its own value.
    q, k, v = (randn((50000, 2, 64), BF, s) for s in (1, 2, 3))
    assert torch.equal(bd.prefill_attn(q, k, v, offsets([1] * 50000)), v)


def test_prefill_sequences_never_see_each_other():
    # The middle sequence holds NaN and infinities in its keys and values.
    d, h, lens = 128, 2, [100, 60, 77]
    q, k, v = (randn((sum(lens), h, d), BF, s) for s in (1, 2, 3))
    k[100:160], v[100:160] = math.inf, math.nan
    for causal in (True, False):
        o = bd.prefill_attn(q, k, v, offsets(lens), causal=causal)
        for a, n in ((0, 100), (160, 77)):
            ro, _, ob, _ = attend(f64(q[a:a + n]), f64(k[a:a + n]), f64(v[a:a + n]), BF, causal)
            check(f64(o[a:a + n]), ro, ob, "a clean sequence")


def test_prefill_keys_hidden_by_the_mask_may_hold_anything():
    # Keys (not values) of hidden positions: infinities, NaN, the type's lowest.
    d, n = 128, 200
    q, k, v = (randn((n, 2, d), BF, s) for s in (1, 2, 3))
    k[150], k[170], k[180] = math.nan, math.inf, torch.finfo(BF).min
    o = bd.prefill_attn(q, k, v, offsets([n]), causal=True)
    ro, _, ob, _ = attend(f64(q[:150]), f64(k[:150]), f64(v[:150]), BF, True)
    check(f64(o[:150]), ro, ob, "rows that do not see them")


@pytest.mark.parametrize("hq,hkv,d", [(8, 2, 128), (3, 1, 128), (8, 8, 64)])
def test_prefill_many_short_sequences(hq, hkv, d):
    # Several items a CTA, empty sequences among them.
    lens = np.random.default_rng(hq).integers(0, 40, 300).tolist()
    run_prefill(BF, d, hq, hkv, lens, lens, True, None, 0.0, False, extra=3)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prefill_rows_behind_the_first_2_to_31_elements(dtype):
    # A row stride of 2^17 elements: the last rows start past 2^31 elements.
    n, d, doc = 16500, 64, 100
    wide = torch.empty((n, 2 ** 17 // d, d), dtype=dtype, device="cuda")
    q, k, v = wide[:, :4], wide[:, 4:6], wide[:, 6:8]
    wide[:, :8] = randn((n, 8, d), dtype, 1)
    assert (n - doc) * wide.stride(0) > 2 ** 31
    o = bd.prefill_attn(q, k, v, offsets([doc] * (n // doc)))
    for a in (0, n - doc):
        ro, _, ob, _ = attend(f64(q[a:a + doc]), f64(k[a:a + doc]), f64(v[a:a + doc]), dtype, True)
        check(f64(o[a:a + doc]), ro, ob, f"O of rows {a}..")


@pytest.mark.parametrize("cap", [0.0, 1.0])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_visible_nan_shows_in_every_row_that_sees_it(dtype, cap):
    n, d, at = 200, 64, 50
    q, k, v = (randn((n, 2, d), dtype, s) for s in (1, 2, 3))
    k[at] = math.nan
    o, lse = bd.prefill_attn(q, k, v, offsets([n]), softcap=cap, with_lse=True)
    assert o[at:].isnan().all() and lse[at:].isnan().all()
    assert not o[:at].isnan().any() and not lse[:at].isnan().any()
    table, pages = make_table([n], 16, 0)
    cache = bd.alloc_paged_cache(pages, 2, 16, d, dtype, "cuda")
    bd.paged_append(k, v, cache, table, offsets([n]), i32([0]))
    for m in (at, n):
        o, lse = bd.paged_attn(q[None, m - 1:m], cache, table, i32([m]), softcap=cap, with_lse=True)
        assert o.isnan().all() == (m > at) and lse.isnan().all() == (m > at)


@pytest.mark.parametrize("cap,bias", [(0.0, False), (20.0, False), (0.0, True), (20.0, True)])
def test_the_only_visible_key_has_weight_one(cap, bias):
    # Its value comes back bit for bit: no rounding of the weight stays in O.
    n, h, d = 70, 3, 128
    q, k, v = (randn((n, h, d), BF, s) for s in (1, 2, 3))
    slopes = slope_list(h) if bias else None
    o = bd.prefill_attn(q, k, v, offsets([1] * n), softcap=cap, slopes=slopes)
    assert torch.equal(o, v)
    table, pages = make_table([1] * n, 16, 0)
    cache = bd.alloc_paged_cache(pages, h, 16, d, BF, "cuda")
    bd.paged_append(k, v, cache, table, offsets([1] * n), i32([0] * n))
    o = bd.paged_attn(q[:, None], cache, table, i32([1] * n), softcap=cap, slopes=slopes)
    assert torch.equal(o[:, 0], v)


@pytest.mark.parametrize("offs", [[0, 40, 20, 60], [0, 30, 90], [-5, 30]])
def test_prefill_bad_offsets_are_flagged(offs):
    q, k, v = (randn((60, 1, 64), BF, s) for s in (1, 2, 3))
    ws = bd.alloc_status_workspace("cuda")
    bd.prefill_attn(q, k, v, i32(offs), ws=ws)
    assert bd.read_device_status(ws) == bd.DEV_BAD_INDEX


# ------------------------------------------------------------------ as used together
def test_serving_run_and_the_filtering_path_agree():
    """Prompt in (append + prefill), one generation block (append + paged
    attention), and the filtering path's own attention over the same rotated
    cache: with every prompt row selected it is the paged attention."""
    h, d, n, g, page, dt = 4, 128, 512, 32, 16, BF
    freq = bd.rope_inv_freq(d)
    q, k, v = (randn((n + g, h, d), dt, s) for s in (1, 2, 3))
    table, pages = make_table([n + g], page, 4)
    cache = bd.alloc_paged_cache(pages, h, page, d, dt, "cuda")
    zero = i32([0])
    first = bd.paged_append(k[:n], v[:n], cache, table, offsets([n]), zero, q=q[:n],
                            inv_freq=freq, keep_keys=True)
    o1 = bd.prefill_attn(first["Q"], first["K"], v[:n], offsets([n]), causal=False)
    ro, _, ob, _ = attend(f64(first["Q"]), f64(first["K"]), f64(v[:n]), dt, False)
    check(f64(o1), ro, ob, "prompt attention")
    block = bd.paged_append(k[n:], v[n:], cache, table, offsets([g]), i32([n]), q=q[n:],
                            inv_freq=freq, keep_keys=True)
    o2, lse2 = bd.paged_attn(block["Q"][None], cache, table, i32([n + g]), causal=False,
                             with_lse=True)
    keys = torch.cat([first["K"], block["K"]])
    ro, rl, ob, lb = attend(f64(block["Q"]), f64(keys), f64(v), dt, False)
    check(f64(o2[0]), ro, ob, "block attention")
    check(f64(lse2[0]), rl, lb, "block lse")
    # The dense cache of the filtering path from the same rotated keys.
    dense = bd.cache_init(keys[None].contiguous(), v[None].contiguous(), n, 3)
    qh = block["Q"].transpose(0, 1)[None].contiguous()
    idx = torch.arange(n, dtype=torch.int32, device="cuda").expand(1, h, n).contiguous()
    o3, lse3 = bd.sparse_gather_attn(qh, dense["Kp"], dense["Vp"], dense["Kg"], dense["Vg"], idx, 3,
                                     bd.alloc_status_workspace("cuda"), with_lse=True)
    assert (o3[0].transpose(0, 1) - o2[0].float()).abs().max() < 2e-2
    assert (lse3[0].t() - lse2[0]).abs().max() < 1e-3


def test_captured_run_replays_with_new_lengths():
    """A decoding step captured once and replayed as the cache grows: lengths
    are device data, so the same graph serves every step."""
    s, hq, hkv, d, page, steps = 3, 8, 2, 128, 16, 20
    start = [1, 15, 100]
    table, pages = make_table([n + steps for n in start], page, 1)
    cache = bd.alloc_paged_cache(pages, hkv, page, d, BF, "cuda")
    for x in cache.values():
        x.zero_()
    hist_k = [randn((n, hkv, d), BF, 10 + i) for i, n in enumerate(start)]
    hist_v = [randn((n, hkv, d), BF, 20 + i) for i, n in enumerate(start)]
    bd.paged_append(torch.cat(hist_k), torch.cat(hist_v), cache, table, offsets(start),
                    i32([0] * s))
    q, k, v = (torch.zeros((s, h, d), dtype=BF, device="cuda") for h in (hq, hkv, hkv))
    cu, held, lens = offsets([1] * s), i32(start), i32([n + 1 for n in start])
    ws = bd.alloc_paged_attn_workspace(q[:, None], cache, table)
    o = torch.empty((s, 1, hq, d), dtype=BF, device="cuda")

    def step():
        bd.paged_append(k, v, cache, table, cu, held)
        bd.paged_attn(q[:, None], cache, table, lens, ws, out=o)
        held.add_(1)
        lens.add_(1)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for t in range(steps):
        for x, seed in ((q, 100), (k, 200), (v, 300)):
            x.copy_(randn(x.shape, BF, seed + t))
        graph.replay()
        hist_k = [torch.cat([a, k[i:i + 1]]) for i, a in enumerate(hist_k)]
        hist_v = [torch.cat([a, v[i:i + 1]]) for i, a in enumerate(hist_v)]
        for i in range(s):
            ro, _, ob, _ = attend(f64(q[i:i + 1]), f64(hist_k[i]), f64(hist_v[i]), BF, True)
            check(f64(o[i]), ro, ob, f"step {t}, sequence {i}")


def test_streams_and_two_calls_at_once():
    args = run_paged(BF, 64, 4, 2, 16, [3000, 500], 1, True, None, 0.0, False)[2]
    q, cache, table, lens, ws = args
    ref = bd.paged_attn(*args)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for _ in range(5):
        for st in streams:
            outs.append(bd.paged_attn(q, cache, table, lens, stream=st))   # own workspaces
    torch.cuda.synchronize()
    assert all(torch.equal(ref, x) for x in outs)
    x, cu = randn((1500, 8, 64), BF, 9), offsets([900, 600])
    ref = bd.prefill_attn(x, x[:, :4], x[:, 4:], cu)
    torch.cuda.synchronize()
    outs = [bd.prefill_attn(x, x[:, :4], x[:, 4:], cu, stream=st) for _ in range(5)
            for st in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(ref, x) for x in outs)


def test_two_captured_graphs_share_a_workspace():
    # Replayed in turn (never at once): each leaves nothing the other minds.
    runs = [run_paged(BF, 128, 8, 2, 16, lens, new, True, None, 0.0, False, seed=new)
            for lens, new in (([900, 40], 1), ([33, 2000], 3))]
    sizes = [r[2][4].numel() for r in runs]
    ws = runs[int(sizes[1] > sizes[0])][2][4]
    graphs = []
    for o, _, (q, cache, table, lens, _) in runs:
        out = torch.zeros_like(o)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            bd.paged_attn(q, cache, table, lens, ws, out=out)
        graphs.append((graph, out, o))
    for _ in range(3):
        for graph, out, ref in graphs:
            out.fill_(7.0)
            graph.replay()
            assert torch.equal(out, ref)


def test_captured_prompt_replays_with_new_offsets():
    h, d, n = 4, 128, 500
    q, k, v = (randn((n, h, d), BF, s) for s in (1, 2, 3))
    cu, out = offsets([n, 0, 0]), torch.empty((n, h, d), dtype=BF, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        bd.prefill_attn(q, k, v, cu, out=out)
    for lens in ([n, 0, 0], [100, 300, 100], [1, 0, 2]):
        cu.copy_(offsets(lens))
        out.fill_(7.0)
        graph.replay()
        assert torch.equal(out[:sum(lens)], bd.prefill_attn(q, k, v, offsets(lens))[:sum(lens)])
        assert (out[sum(lens):] == 7).all()


def test_binding_refuses_what_the_kernels_do_not_take():
    d, page = 64, 16
    k, v, q = (randn((6, h, d), BF, h) for h in (2, 2, 4))
    cache = bd.alloc_paged_cache(4, 2, page, d, BF, "cuda")
    table, cu, held = i32([[0, 1], [2, 3]]), i32([0, 3, 6]), i32([0, 0])
    ok = dict(k=k, v=v, cache=cache, page_table=table, cu_rows=cu, cache_len=held)
    for bad in (dict(k=k.float()), dict(v=v[:5]), dict(k=k.cpu()), dict(v=v.cpu()),
                dict(k=k.transpose(1, 2).contiguous().transpose(1, 2)), dict(cu_rows=cu[:2]),
                dict(cu_rows=cu.long()), dict(cache_len=held.cpu()), dict(page_table=table.t()),
                dict(positions=i32([0] * 5)), dict(q=q, out={"Q": q[:5]}),
                dict(cache={"K": cache["K"], "V": cache["V"][:3]})):
        with pytest.raises(ValueError):
            bd.paged_append(**{**ok, **bad})
    half = {n: x.half() for n, x in cache.items()}
    with pytest.raises(ValueError):
        bd.paged_append(**{**ok, "k": k.half(), "v": v.half(), "cache": half})
    lens = i32([3, 3])
    ok = dict(q=q[:2, None], cache=cache, page_table=table, kv_len=lens)
    for bad in (dict(q=q[:2]), dict(q=q[:1, None]), dict(kv_len=lens[:1]), dict(scale=0.0),
                dict(prefix=lens.float()), dict(slopes=torch.ones(2, device="cuda")),
                dict(out=torch.empty((2, 1, 4, d), device="cuda"))):
        with pytest.raises(ValueError):
            bd.paged_attn(**{**ok, **bad})
    with pytest.raises(bd.WfError):
        bd.paged_attn(**{**ok, "ws": torch.empty(64, dtype=torch.uint8, device="cuda")})
    with pytest.raises(bd.WfError):
        bd.paged_attn(**{**ok, "softcap": -1.0})
    ok = dict(q=q, k=k, v=v, cu_q=cu)
    for bad in (dict(q=q[None]), dict(v=v[:5]), dict(cu_k=cu[:2]), dict(k=k.expand(6, 2, d).cpu()),
                dict(slopes=torch.ones(3, device="cuda"))):
        with pytest.raises(ValueError):
            bd.prefill_attn(**{**ok, **bad})
    for bad in (dict(q=q[:, :3]), dict(k=k[:1].expand(6, 2, d), v=v), dict(scale=-1.0)):
        with pytest.raises((ValueError, bd.WfError)):
            bd.prefill_attn(**{**ok, **bad})

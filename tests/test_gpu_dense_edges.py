"""GPU checks of calls at the edges of the paged append and the dense
attentions: positions that fp32 does not hold, what follows a call in a graph,
visible infinities and largest values, tables of high frequencies, extreme
scales and caps."""

import math

import numpy as np
import pytest
import torch

from dense_common import attend, check, f64, half_step, rotation_bound
from test_gpu_dense_attn import BF, F32, i32, make_table, offsets, randn, slope_list
from wavelet_guided_sparse_gb300 import binding as bd

pytestmark = pytest.mark.gpu


def one_cache(k, v, page=16, seed=0):
    """A paged cache holding one sequence's rows k, v [n, hkv, d], and its table."""
    n, hkv, d = k.shape
    table, pages = make_table([n], page, seed)
    cache = bd.alloc_paged_cache(pages, hkv, page, d, k.dtype, "cuda")
    bd.paged_append(k, v, cache, table, offsets([n]), i32([0]))
    return cache, table


@pytest.mark.parametrize("dtype,cap,new", [(BF, 0.0, 1), (BF, 30.0, 3), (F32, 0.0, 2)])
def test_paged_bias_counts_distances_past_2_to_24(dtype, cap, new):
    # A cache of more than 2^24 rows: one page repeated, but for a window of
    # distinct pages at its end.  Rows before the window weigh e^-400 at most.
    page, d, n, tail = 256, 64, 2 ** 24 + 65, 17
    need = -(-n // page)
    table = torch.zeros((1, need), dtype=torch.int32, device="cuda")
    table[0, -tail:] = torch.arange(1, tail + 1, dtype=torch.int32)
    cache = {x: randn((tail + 1, 1, page, d), dtype, s) for s, x in enumerate(("K", "V"))}
    slopes = torch.tensor([0.84, 0.5, 0.25, 0.1], device="cuda")
    q = randn((1, new, 4, d), dtype, 5)
    o, lse = bd.paged_attn(q, cache, table, i32([n]), softcap=cap, slopes=slopes, with_lse=True)
    w = n - (need - tail) * page
    k, v = (f64(cache[x][1:]).reshape(-1, 1, d)[:w] for x in ("K", "V"))
    ro, rl, ob, lb = attend(f64(q[0]), k, v, dtype, True, 0, cap, slopes.cpu().numpy())
    check(f64(lse[0]), rl, lb, "lse")
    check(f64(o[0]), ro, ob, "O")


@pytest.mark.parametrize("lens", [[0] * 7, [1 + i % 64 for i in range(2000)], [64] * 38])
def test_what_follows_in_a_graph_sees_finished_outputs(lens):
    # Contexts of at most one tile: no unit is split, so nothing is left to the
    # joining launch, and the nodes behind it read and overwrite at once.
    hq, hkv, d, page = 8, 4, 128, 32
    s = len(lens)
    table, pages = make_table([64] * s, page, 3)
    cache = {x: randn((pages, hkv, page, d), BF, i) for i, x in enumerate(("K", "V"))}
    q = randn((s, 1, hq, d), BF, 4)
    ws = bd.alloc_paged_attn_workspace(q, cache, table)
    first, held = i32(lens), i32(lens)
    ref, ref_lse = bd.paged_attn(q, cache, table, first, ws, with_lse=True)
    torch.cuda.synchronize()
    o, seen = torch.empty_like(ref), torch.empty_like(ref)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        held.copy_(first)
        bd.paged_attn(q, cache, table, held, ws, out=o)
        held.add_(1)
        seen.copy_(o)
        o.fill_(7.0)
    for _ in range(50):
        seen.fill_(7.0)
        graph.replay()
        assert torch.equal(seen, ref) and torch.equal(held, first + 1)
    if s == 7:
        assert (ref == 0).all() and (ref_lse == -math.inf).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_paged_largest_values_behind_a_lower_maximum(dtype):
    # The key of the largest value scores 5 above all others, far behind them: its
    # weight must not exceed 1 on the way.  Many tiles a CTA: 64 like sequences.
    s, h, d, n, at = 64, 4, 64, 700, 690
    q, k, v = torch.zeros((s, 1, h, d), device="cuda"), torch.zeros((n, h, d), device="cuda"), \
        randn((n, h, d), F32, 1)
    q[..., 0] = 1.0
    k[at, :, 0] = 5.0 * math.sqrt(d)
    v[at, :, 1] = 3e38
    q, k, v = q.to(dtype), k.to(dtype), v.to(dtype)
    cache, table = one_cache(k, v)
    o, lse = bd.paged_attn(q, cache, table.expand(s, -1).contiguous(), i32([n] * s), with_lse=True)
    ro, rl, ob, lb = attend(f64(q[0]), f64(k), f64(v), dtype, True)
    for i in range(s):
        check(f64(lse[i]), rl, lb, "lse")
        check(f64(o[i]), ro, ob, "O")


@pytest.mark.parametrize("at", [0, 150, 299])
@pytest.mark.parametrize("dtype,cap,bias", [(BF, 0.0, False), (BF, 50.0, False), (BF, 0.0, True),
                                            (F32, 0.0, False)])
def test_prefill_largest_values_behind_a_lower_maximum(dtype, cap, bias, at):
    n, h, d = 300, 2, 128
    q, k, v = torch.zeros((n, h, d), device="cuda"), torch.zeros((n, h, d), device="cuda"), \
        randn((n, h, d), F32, 1)
    q[..., 0] = 1.0
    k[at, :, 0] = 5.0 * math.sqrt(d)
    v[at, :, 1] = 3e38
    q, k, v = q.to(dtype), k.to(dtype), v.to(dtype)
    slopes = torch.zeros(h, device="cuda") if bias else None
    o, lse = bd.prefill_attn(q, k, v, offsets([n]), causal=False, softcap=cap, slopes=slopes,
                             with_lse=True)
    ro, rl, ob, lb = attend(f64(q), f64(k), f64(v), dtype, False, 0, cap)
    check(f64(lse), rl, lb, "lse")
    check(f64(o), ro, ob, "O")


@pytest.mark.parametrize("d,hq,hkv,new", [(64, 2, 2, 1), (128, 4, 1, 16), (128, 8, 2, 5),
                                          (128, 8, 1, 4)])
def test_paged_fp32_visible_infinities_and_largest_values(d, hq, hkv, new):
    n, big = 300, torch.finfo(F32).max
    q, k, v = randn((1, new, hq, d), F32, 1), randn((n, hkv, d), F32, 2), randn((n, hkv, d), F32, 3)
    q[..., 3] = -q[..., 3].abs() - 0.5
    k[40, :, 3] = math.inf                    # score -inf: weight 0
    tiny = 2.0 ** -124
    q[..., 5] = tiny
    k[100], k[150] = 0.0, 0.0
    k[100, :, 5], k[150, :, 5] = big, -big    # scores of +-16 / sqrt(d)
    v[7, :, 2], v[9, :, 4] = big, math.inf
    cache, table = one_cache(k, v)
    o, lse = bd.paged_attn(q, cache, table, i32([n]), causal=False, with_lse=True)
    # The same products with channel 5 at ordinary size, without the key of weight 0
    # (scaling by powers of two changes no rounding).
    keep = np.arange(n) != 40
    qr, kr, vr = f64(q[0]), f64(k)[keep], f64(v)[keep]
    qr[..., 5], kr[..., 5] = 1.0, kr[..., 5] * tiny
    vr[..., 4] = 0.0
    ro, rl, ob, lb = attend(qr, kr, vr, F32, False)
    rest = np.arange(d) != 4
    check(f64(lse[0]), rl, lb, "lse")
    check(f64(o[0])[..., rest], ro[..., rest], ob[..., rest], "O")
    assert (o[0, ..., 4] == math.inf).all()


@pytest.mark.parametrize("hq,new", [(1, 1), (4, 5), (8, 8)])
def test_paged_fp32_capped_scores_of_an_infinite_query(hq, new):
    # Its scores are the cap, either way: two weights, e^cap and e^-cap.
    n, d, cap = 200, 64, 3.0
    q, k, v = randn((1, new, hq, d), F32, 1), randn((n, 1, d), F32, 2), randn((n, 1, d), F32, 3)
    q[..., 9] = math.inf
    k[..., 9] += torch.where(k[..., 9] < 0, -0.1, 0.1)
    cache, table = one_cache(k, v)
    o, lse = bd.paged_attn(q, cache, table, i32([n]), causal=False, softcap=cap, with_lse=True)
    z = cap * np.sign(f64(k)[:, 0, 9])
    p = np.exp(z) / np.exp(z).sum()
    ref, a = p @ f64(v)[:, 0], p @ np.abs(f64(v)[:, 0])
    # tanh, scaling and the log2 domain: cap (2^-20 + 8 2^-24) of a score, twice; 2^x
    # 2^-20; the sum of n terms n 2^-24; the last rounding.
    ez = cap * (2.0 ** -20 + 2.0 ** -21)
    bound = a * (2 * ez + 2.0 ** -20 + n * 2.0 ** -24) * 1.01 + 2.0 ** -24 * (np.abs(ref) + a)
    rl = math.log(np.exp(z).sum())
    check(f64(o[0]), np.broadcast_to(ref, (new, hq, d)), bound, "O")
    check(f64(lse[0]), np.full((new, hq), rl), ez + 2.0 ** -20 + 2.0 ** -22 * abs(rl), "lse")


@pytest.mark.parametrize("dtype,d,hq,inter,t", [(BF, 128, 8, False, 700), (BF, 64, 4, True, 33),
                                                (F32, 64, 2, False, 1), (F32, 128, 6, True, 900)])
def test_append_in_place_queries_are_those_out_of_place(dtype, d, hq, inter, t):
    page, hkv = 16, 2
    q, k, v = randn((t, hq, d), dtype, 1), randn((t, hkv, d), dtype, 2), randn((t, hkv, d), dtype, 3)
    table, pages = make_table([t + 3], page, 0)
    cache = bd.alloc_paged_cache(pages, hkv, page, d, dtype, "cuda")
    call = dict(inv_freq=bd.rope_inv_freq(d), interleaved=inter)
    args = (k, v, cache, table, offsets([t]), i32([3]))
    ref = bd.paged_append(*args, q=q, **call)["Q"]
    assert bd.paged_append(*args, q=q, out={"Q": q}, **call)["Q"] is q
    assert torch.equal(q, ref)


def test_append_turns_by_high_frequencies_at_far_positions():
    # Whole-number frequencies, so that the angle of a position is exact in 64 bits.
    # The bound is that of any rotation: the reduction adds nothing to it.
    d, h, pos = 64, 2, [2 ** 31 - 1, 2 ** 30 + 12345, 10 ** 9 + 7, -10 ** 9, 3]
    t = len(pos)
    freq = [1000.0 - 7 * i for i in range(30)] + [1.0, 2.0]
    x = randn((t, h, d), F32, 1)
    table, pages = make_table([t], 8, 0)
    cache = bd.alloc_paged_cache(pages, h, 8, d, F32, "cuda")
    got = bd.paged_append(x, x, cache, table, offsets([t]), i32([0]), inv_freq=freq,
                          positions=i32(pos), keep_keys=True)["K"]
    ref, a = np.empty((t, h, d)), f64(x)
    for i, p in enumerate(pos):
        for j, f in enumerate(freq):
            c, s = math.cos(p * f), math.sin(p * f)
            ref[i, :, j] = a[i, :, j] * c - a[i, :, j + 32] * s
            ref[i, :, j + 32] = a[i, :, j] * s + a[i, :, j + 32] * c
    check(f64(got), ref, rotation_bound(a, d, False, ref, F32), "keys")


@pytest.mark.parametrize("cap,scale", [(1e-38, None), (0.0, 1e-38), (1e30, None)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_bias_beside_extreme_scales_and_caps(dtype, cap, scale):
    # Scores that vanish beside the bias (or meet an ordinary one under a far cap).
    d, n, h = 128, 200, 2
    q, k, v = (randn((n, h, d), dtype, s) for s in (1, 2, 3))
    slopes = torch.tensor([0.5, 0.03125], device="cuda")
    sl = slopes.cpu().numpy()
    bend = min(cap, 20.0) if cap else None
    ro, rl, ob, lb = attend(f64(q), f64(k), f64(v), dtype, True, 0, cap, sl, scale, bend=bend)
    o, lse = bd.prefill_attn(q, k, v, offsets([n]), softcap=cap, scale=scale, slopes=slopes,
                             with_lse=True)
    check(f64(lse), rl, lb, "lse")
    check(f64(o), ro, ob, "O")
    cache, table = one_cache(k, v)
    o, lse = bd.paged_attn(q[None, -9:], cache, table, i32([n]), softcap=cap, scale=scale,
                           slopes=slopes, with_lse=True)
    check(f64(lse[0]), rl[-9:], lb[-9:], "lse over pages")
    check(f64(o[0]), ro[-9:], ob[-9:], "O over pages")


@pytest.mark.parametrize("scale,low,top,value", [
    (0.5584592656208399, 1.234375, 13.375, 1.25), (0.4848162855389709, 1.421875, 15.625, 1.4375),
    (0.47954654330485164, 1.4375, 12.875, 1.5), (0.4644029682531195, 1.484375, 13.375, 1.6875)])
def test_prefill_weights_meet_one_rounding(scale, low, top, value):
    # 95 like weights just short of a rounding midpoint, and behind them in the same
    # tile one key that outweighs them by 2^8 to 2^11: rounded once more when they are
    # rescaled (or by a factor that is itself rounded), they leave the bound.
    h, d, n = 2, 128, 97
    q, k, v = (torch.zeros((n, h, d), device="cuda") for _ in range(3))
    q[..., 0] = 1.0
    k[1:96, :, 0], k[96, :, 0] = -low, top
    v[1:96] = value
    q, k, v = q.to(BF), k.to(BF), v.to(BF)
    o, lse = bd.prefill_attn(q, k, v, offsets([n]), causal=False, scale=scale,
                             slopes=torch.zeros(h, device="cuda"), with_lse=True)
    ro, rl, ob, lb = attend(f64(q), f64(k), f64(v), BF, False, scale=float(np.float32(scale)))
    check(f64(lse), rl, lb, "lse")
    check(f64(o), ro, ob, "O")


def test_append_returns_what_it_wrote():
    k, v = randn((4, 2, 64), BF, 1), randn((4, 2, 64), BF, 2)
    cache = bd.alloc_paged_cache(1, 2, 16, 64, BF, "cuda")
    spare = {x: torch.empty((4, 2, 64), dtype=BF, device="cuda") for x in ("Q", "K")}
    args = (k, v, cache, i32([[0]]), offsets([4]), i32([0]))
    assert bd.paged_append(*args, out=spare) == {}
    res = bd.paged_append(*args, out=spare, keep_keys=True)
    assert set(res) == {"K"} and res["K"] is spare["K"] and torch.equal(res["K"], k)


def test_paged_workspace_refuses_queries_without_a_block_axis():
    q = randn((2, 4, 64), BF, 1)
    cache = bd.alloc_paged_cache(2, 2, 16, 64, BF, "cuda")
    for bad in (q, q[0], q[None, :, None]):
        with pytest.raises(ValueError):
            bd.alloc_paged_attn_workspace(bad, cache, i32([[0], [1]]))


@pytest.mark.parametrize("dtype,new,lens", [(BF, 1, [40]), (BF, 1, [9000, 30000, 70]), (BF, 64, [200]),
                                            (BF, 9, [5000] * 40), (F32, 1, [64, 64]),
                                            (F32, 16, [3000] * 30)])
def test_paged_wait_that_runs_out_is_reported_and_recovers(dtype, new, lens):
    # The first tile's copies of the first CTA are never issued (nothing else is in
    # flight when its wait gives up, or it is waited for): the call ends, says so,
    # and the next one is as before.
    page, hq, hkv, d = 64, 4, 2, 128
    table, pages = make_table(lens, page, 1)
    cache = {x: randn((pages, hkv, page, d), dtype, i) for i, x in enumerate(("K", "V"))}
    q, n = randn((len(lens), new, hq, d), dtype, 3), i32(lens)
    ws = bd.alloc_paged_attn_workspace(q, cache, table)
    ref, lse = bd.paged_attn(q, cache, table, n, ws, with_lse=True)
    assert bd.read_device_status(ws) == 0
    bd.inject_wait_timeout(1000)
    bd.paged_attn(q, cache, table, n, ws)
    bd.inject_wait_timeout(0)
    assert bd.read_device_status(ws) == bd.DEV_WAIT_TIMEOUT    # synchronises
    bd.clear_device_status(ws)
    o, lse2 = bd.paged_attn(q, cache, table, n, ws, with_lse=True)
    assert bd.read_device_status(ws) == 0
    assert torch.equal(o, ref) and torch.equal(lse, lse2)


@pytest.mark.parametrize("d,hq,lens,cap", [(128, 4, [100], 0.0), (64, 3, [2000, 5, 700], 20.0),
                                           (128, 8, [6000, 1000], 0.0), (64, 2, [90] * 400, 0.0)])
def test_prefill_wait_that_runs_out_is_reported_and_recovers(d, hq, lens, cap):
    q, k, v = (randn((sum(lens), hq, d), BF, s) for s in (1, 2, 3))
    cu, ws = offsets(lens), bd.alloc_status_workspace("cuda")
    ref, lse = bd.prefill_attn(q, k, v, cu, softcap=cap, with_lse=True, ws=ws)
    assert bd.read_device_status(ws) == 0
    bd.inject_wait_timeout(1000)
    bd.prefill_attn(q, k, v, cu, softcap=cap, ws=ws)
    bd.inject_wait_timeout(0)
    assert bd.read_device_status(ws) == bd.DEV_WAIT_TIMEOUT
    bd.clear_device_status(ws)
    o, lse2 = bd.prefill_attn(q, k, v, cu, softcap=cap, with_lse=True, ws=ws)
    assert bd.read_device_status(ws) == 0
    assert torch.equal(o, ref) and torch.equal(lse, lse2)


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("cap,scale,spread", [(1e-2, 50.0, 3e-5), (1e-2, 2.0, 5e-4), (2e3, 1.0, 40.0)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_small_and_large_caps_form_the_scores(dtype, cap, scale, spread, bias):
    # Scores about the cap's bend, of a size that the lse shows: its bound is far
    # below them (small caps), or they decide the row (large ones).
    d, n, h = 128, 200, 2
    q, k, v = (randn((n, h, d), dtype, s) for s in (1, 2, 3))
    q = (q.float() * spread).to(dtype)
    slopes = torch.tensor([cap / 100, cap / 1000], device="cuda") if bias else None
    sl = None if slopes is None else slopes.cpu().numpy()
    ro, rl, ob, lb = attend(f64(q), f64(k), f64(v), dtype, True, 0, cap, sl, scale)
    flat = np.log(np.arange(1, n + 1))[:, None]          # the lse of scores of 0
    assert np.median(np.abs(rl - flat) / lb) > 20
    o, lse = bd.prefill_attn(q, k, v, offsets([n]), softcap=cap, scale=scale, slopes=slopes,
                             with_lse=True)
    check(f64(lse), rl, lb, "lse")
    check(f64(o), ro, ob, "O")
    cache, table = one_cache(k, v)
    o, lse = bd.paged_attn(q[None, -9:], cache, table, i32([n]), softcap=cap, scale=scale,
                           slopes=slopes, with_lse=True)
    check(f64(lse[0]), rl[-9:], lb[-9:], "lse over pages")
    check(f64(o[0]), ro[-9:], ob[-9:], "O over pages")


@pytest.mark.parametrize("cap,bias", [(0.0, False), (20.0, False), (0.0, True), (20.0, True)])
def test_bf16_visible_infinities_and_largest_values(cap, bias):
    d, h, n, big, tiny = 128, 4, 300, torch.finfo(BF).max, 2.0 ** -124
    q, k, v = (randn((n, h, d), BF, s) for s in (1, 2, 3))
    q[..., 3] = -q[..., 3].abs() - 0.5
    q[..., 5] = tiny
    k[100], k[150] = 0.0, 0.0
    k[100, :, 5], k[150, :, 5] = big, -big    # scores of +-16 / sqrt(d)
    v[7, :, 2], v[9, :, 4] = big, math.inf
    keep = np.ones(n, bool)
    if cap == 0.0 and not bias:
        k[40, :, 3], keep[40] = math.inf, False       # a score of -inf: weight 0
    slopes = slope_list(h) / 16 if bias else None
    # The same products with channel 5 at ordinary size, without the key of weight 0.
    qr, kr, vr = f64(q), f64(k)[keep], f64(v)[keep]
    qr[..., 5], kr[..., 5], vr[..., 4] = 1.0, kr[..., 5] * tiny, 0.0
    rest = np.arange(d) != 4
    o, lse = bd.prefill_attn(q, k, v, offsets([n]), causal=False, softcap=cap, slopes=slopes,
                             with_lse=True)
    ro, rl, ob, lb = attend(qr, kr, vr, BF, False, 0, cap,
                            None if slopes is None else slopes.cpu().numpy())
    check(f64(lse), rl, lb, "lse")
    check(f64(o)[..., rest], ro[..., rest], ob[..., rest], "O")
    assert (o[..., 4] == math.inf).all()
    cache, table = one_cache(k, v)
    o, lse = bd.paged_attn(q[None, -9:], cache, table, i32([n]), causal=False, softcap=cap,
                           slopes=slopes, with_lse=True)
    check(f64(lse[0]), rl[-9:], lb[-9:], "lse over pages")
    check(f64(o[0])[..., rest], ro[-9:][..., rest], ob[-9:][..., rest], "O over pages")
    assert (o[0, ..., 4] == math.inf).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prefill_without_any_key(dtype):
    q, none = randn((70, 4, 64), dtype, 1), torch.empty((0, 2, 64), dtype=dtype, device="cuda")
    for causal in (True, False):
        o, lse = bd.prefill_attn(q, none, none, offsets([50, 20]), offsets([0, 0]), causal=causal,
                                 with_lse=True)
        assert (o == 0).all() and (lse == -math.inf).all()
    o, lse = bd.prefill_attn(q[:0], none, none, offsets([0]), with_lse=True)
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)


@pytest.mark.parametrize("d,hq,hkv,new,n,cap,bias", [
    (128, 8, 2, 1, 900, 0.0, False), (128, 4, 4, 1, 5000, 20.0, True), (64, 16, 1, 1, 333, 0.0, True),
    (64, 4, 1, 4, 2000, 0.0, False), (128, 2, 2, 5, 700, 30.0, False)])
def test_paged_up_to_16_rows_only_the_output_is_rounded(d, hq, hkv, new, n, cap, bias):
    # Weights in two bf16 parts are good to 2^-15: what is left are fp32's roundings
    # (attend()'s bound at that type) and the output's half a step.
    q = randn((1, new, hq, d), BF, 1)
    k, v = randn((n, hkv, d), BF, 2), randn((n, hkv, d), BF, 3)
    slopes = slope_list(hq) if bias else None
    cache, table = one_cache(k, v)
    o = bd.paged_attn(q, cache, table, i32([n]), softcap=cap, slopes=slopes)
    args = (F32, True, 0, cap, None if slopes is None else slopes.cpu().numpy())
    ro, _, ob, _ = attend(f64(q[0]), f64(k), f64(v), *args)
    ra = attend(f64(q[0]), f64(k), np.abs(f64(v)), *args)[0]
    inner = ob + ra * 2.0 ** -15 * 1.01
    check(f64(o[0]), ro, inner + half_step(BF) * (np.abs(ro) + inner), "O")


@pytest.mark.parametrize("inter", [False, True])
def test_append_sines_and_cosines_are_good_to_their_last_places(inter):
    # Pairs (1, 0) become the cosine and the sine themselves.  Two units of each
    # (2^-23, twice that beside the correction for the angle's last bits), and what
    # the correction's own roundings leave where a value is near 0: 2^-24 of 2^-24.
    d, t = 64, 4000
    freq = list(bd.rope_inv_freq(d, 10000.0))
    pos = np.random.default_rng(1).integers(0, 2 ** 20, t)
    pos[:7] = [0, 1, 22, 333, 355, 103993, 104348]      # 355: 113 half turns and 3e-5
    x = torch.zeros((t, 1, d), device="cuda")
    x[..., slice(0, d, 2) if inter else slice(0, d // 2)] = 1.0
    cache = bd.alloc_paged_cache(-(-t // 256), 1, 256, d, F32, "cuda")
    table = torch.arange(-(-t // 256), dtype=torch.int32, device="cuda")[None]
    got = f64(bd.paged_append(x, x, cache, table, offsets([t]), i32([0]), inv_freq=freq,
                              interleaved=inter, positions=i32(pos.tolist()), keep_keys=True)["K"])[:, 0]
    cs, sn = (got[:, 0::2], got[:, 1::2]) if inter else (got[:, :d // 2], got[:, d // 2:])
    # The reference's own product p f rounds by 2^-53 of it.
    a = pos[:, None] * np.asarray(freq)[None]
    for g, ref in ((cs, np.cos(a)), (sn, np.sin(a))):
        err = np.abs(g - ref)
        bound = 2.0 ** -22 * np.abs(ref) + 2.0 ** -46 + 2.0 ** -53 * np.abs(a)
        assert (err <= bound).all(), (err / bound).max()


@pytest.mark.parametrize("where", ["front", "spread", "back"])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_prefill_padded_batch_is_the_compact_one(dtype, where):
    # Four prompts among 4096 sequences, the rest empty: the same bits, and not the
    # milliseconds that a block for each empty sequence and head would cost.
    lens, slots = [300, 1, 128, 83], 4096
    at = {"front": [0, 1, 2, 3], "spread": [5, 1000, 1001, 4000], "back": [4092, 4093, 4094, 4095]}[where]
    padded = [0] * slots
    for i, n in zip(at, lens):
        padded[i] = n
    q, k, v = (randn((sum(lens), h, 128), dtype, h) for h in (32, 8, 8))
    v = v + 1
    times, outs = [], []
    for cu in (offsets(lens), offsets(padded)):
        ws = bd.alloc_status_workspace("cuda")
        outs.append(bd.prefill_attn(q, k, v, cu, with_lse=True, ws=ws))
        assert bd.read_device_status(ws) == 0
        best = math.inf
        for _ in range(5):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            bd.prefill_attn(q, k, v, cu)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        times.append(best)
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
    assert times[1] < 4 * times[0] + 0.5, times


@pytest.mark.parametrize("dtype,hq,hkv", [(BF, 4, 1), (BF, 3, 3), (F32, 2, 1)])
def test_prefill_more_row_blocks_than_the_grid_takes(dtype, hq, hkv):
    # 40000 sequences of 0 to 3 rows: several row blocks a block of the grid.
    lens = np.random.default_rng(7).integers(0, 4, 40000)
    t, d = int(lens.sum()), 64
    q, k, v = (randn((t, h, d), dtype, s) for s, h in ((1, hq), (2, hkv), (3, hkv)))
    o = bd.prefill_attn(q, k, v, offsets(lens.tolist()))
    first = np.repeat(np.cumsum(lens) - lens, lens)
    pos = torch.arange(t, device="cuda")
    start = torch.tensor(first, device="cuda")
    # Each row sees at most three keys: its own and the two before it.
    z, vals = [], []
    for back in range(3):
        j = (pos - back).clamp(min=0)
        kk = k[j].double().repeat_interleave(hq // hkv, 1)
        zz = (q.double() * kk).sum(-1) / d ** 0.5
        z.append(zz.masked_fill((pos - back < start)[:, None], -math.inf))
        vals.append(v[j].double().repeat_interleave(hq // hkv, 1))
    p = torch.softmax(torch.stack(z), 0)
    ref = sum(p[i][..., None] * vals[i] for i in range(3))
    bound = sum(p[i][..., None] * vals[i].abs() for i in range(3))
    # As in attend(): the score's dot product d 2^-23 |q||k|, its other roundings, 2^x;
    # the weights' and the output's one rounding each.
    hs = half_step(dtype)
    big = q.double().norm(dim=-1).max().item() * k.double().norm(dim=-1).max().item() / d ** 0.5
    e = 2 * (d * 2.0 ** -23 * big + 8 * 2.0 ** -24 * 2 * big) + 2.0 ** -20
    bound = bound * (hs + e) * 1.01 + hs * (ref.abs() + bound * (hs + e))
    assert ((o.double() - ref).abs() <= bound).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prefill_checks_the_offsets_of_a_batch_without_rows(dtype):
    q, k, v = (randn((60, 8, 64), dtype, s) for s in (1, 2, 3))
    ws, out = bd.alloc_status_workspace("cuda"), torch.full((60, 8, 64), 7.0, dtype=dtype, device="cuda")
    bd.prefill_attn(q, k, v, i32([0] * 4097), out=out, ws=ws)
    assert bd.read_device_status(ws) == 0 and (out == 7).all()
    bd.prefill_attn(q, k, v, i32([0] * 4096 + [-1]), out=out, ws=ws)
    assert bd.read_device_status(ws) == bd.DEV_BAD_INDEX and (out == 7).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_paged_padded_batch_is_the_compact_one(dtype):
    # Four sequences in front of 4092 idle slots: the same rows, and the idle slots
    # cost no walk of one after the other.
    live, slots, hq, hkv, d, page, n = 4, 4096, 32, 8, 128, 16, 1000
    table, pages = make_table([n] * live, page, 3)
    wide = torch.full((slots, table.shape[1]), -7, dtype=torch.int32, device="cuda")
    wide[:live] = table
    cache = {x: randn((pages, hkv, page, d), dtype, i) for i, x in enumerate(("K", "V"))}
    q = torch.zeros((slots, 1, hq, d), dtype=dtype, device="cuda")
    q[:live] = randn((live, 1, hq, d), dtype, 5)
    lens = i32([n] * live + [0] * (slots - live))
    times, outs = [], []
    for m, t in ((live, table), (slots, wide)):
        ws = bd.alloc_paged_attn_workspace(q[:m], cache, t)
        call = dict(q=q[:m], cache=cache, page_table=t, kv_len=lens[:m], ws=ws)
        outs.append(bd.paged_attn(with_lse=True, **call))
        assert bd.read_device_status(ws) == 0
        best = math.inf
        for _ in range(10):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            bd.paged_attn(**call)
            b.record()
            torch.cuda.synchronize()
            best = min(best, a.elapsed_time(b))
        times.append(best)
    # The work is divided differently: fp32 sums in another order.
    for x, y in zip(outs[0], outs[1]):
        tol = 2 * half_step(dtype) if x.dtype == dtype else 2.0 ** -18
        assert ((x - y[:live]).abs() <= tol * x.abs() + 2.0 ** -18).all()
        assert (y[live:] == (0 if x.dim() == 4 else -math.inf)).all()
    assert times[1] < times[0] + 0.15, times


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (20.0, False), (0.0, True), (20.0, True)])
def test_prefill_what_is_hidden_changes_no_bit(dtype, cap, bias):
    # Keys that the mask hides from the first rows, and all of the next sequence.  (128
    # rows: a capped score's form is chosen for 32 rows at a time, by what these see.)
    d, h, lens, seen = 128, 4, [300, 77, 41], 128
    t = sum(lens)
    q, k, v = (randn((t, h, d), dtype, s) for s in (1, 2, 3))
    slopes = slope_list(h) if bias else None
    outs = []
    for junk in (0.0, 300.0, -1e30, math.nan):
        k[seen:300], k[377:] = junk, junk
        v[377:] = junk
        o, lse = bd.prefill_attn(q, k, v, offsets(lens), softcap=cap, slopes=slopes, with_lse=True)
        outs.append([x[a:b].clone() for x in (o, lse) for a, b in ((0, seen), (300, 377))])
    for other in outs[1:]:
        assert all(torch.equal(x, y) for x, y in zip(other, outs[0]))


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("n", [76, 77, 128 + 45])
def test_prefill_capped_scores_beside_another_sequences_nan(n, bias):
    # Scores far into the cap's bend, and in the next sequence's keys, right behind
    # the last one that counts, NaN.
    d, h, cap = 128, 2, 2.0
    q, k, v = (randn((n + 90, h, d), BF, s) for s in (1, 2, 3))
    q, k[n:], v[n:] = q * 4, math.nan, math.nan
    slopes = slope_list(h) if bias else None
    o, lse = bd.prefill_attn(q, k, v, offsets([n, 90]), softcap=cap, slopes=slopes, with_lse=True)
    ro, rl, ob, lb = attend(f64(q[:n]), f64(k[:n]), f64(v[:n]), BF, True, 0, cap,
                            None if slopes is None else slopes.cpu().numpy())
    check(f64(lse[:n]), rl, lb, "lse")
    check(f64(o[:n]), ro, ob, "O")


@pytest.mark.parametrize("dtype,new", [(BF, 1), (BF, 12), (F32, 1), (F32, 12)])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (20.0, False), (20.0, True)])
def test_paged_what_lies_behind_a_sequence_changes_no_bit(dtype, new, cap, bias):
    page, hq, hkv, d, lens = 64, 4, 2, 128, [50, 90, 1000, 200]
    table, pages = make_table(lens, page, 1)
    cache = {x: randn((pages, hkv, page, d), dtype, i) for i, x in enumerate(("K", "V"))}
    q = randn((len(lens), new, hq, d), dtype, 3)
    slopes = slope_list(hq) if bias else None
    outs = []
    for junk_k, junk_v in ((0.0, 0.0), (1e30, -1e30), (math.nan, math.inf)):
        for s, n in enumerate(lens):
            if n % page:
                last = table[s, n // page]
                cache["K"][last, :, n % page:] = junk_k
                cache["V"][last, :, n % page:] = junk_v
        outs.append(bd.paged_attn(q, cache, table, i32(lens), softcap=cap, slopes=slopes,
                                  with_lse=True))
    for o, lse in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(lse, outs[0][1])


@pytest.mark.parametrize("hq,hkv", [(4, 4), (4, 2)])
@pytest.mark.parametrize("cap,bias", [(0.0, False), (20.0, False), (20.0, True)])
def test_prefill_the_next_sequences_queries_change_no_bit(hq, hkv, cap, bias):
    # They lie in the same query tile as this one's last rows.
    d, lens = 128, [300, 77, 41]
    t = sum(lens)
    q, k, v = randn((t, hq, d), BF, 1), randn((t, hkv, d), BF, 2), randn((t, hkv, d), BF, 3)
    slopes = slope_list(hq) if bias else None
    outs = []
    for junk in (0.0, 300.0, -1e30, math.nan):
        q[377:] = junk
        o, lse = bd.prefill_attn(q, k, v, offsets(lens), softcap=cap, slopes=slopes, with_lse=True)
        outs.append((o[:377].clone(), lse[:377].clone()))
    for o, lse in outs[1:]:
        assert torch.equal(o, outs[0][0]) and torch.equal(lse, outs[0][1])

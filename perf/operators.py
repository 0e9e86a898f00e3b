"""Operators of the paged cache and the dense attentions around the filtering path.

Three operators, as a serving loop uses them:

* append: new rows' keys and values into a paged cache, keys and queries rotated
  to their positions on the way;
* paged: attention of one new token (or one generation block) per sequence over
  that cache;
* prefill: attention of packed prompts over their own keys and values, with a
  document mask, causal and prefix masks, a tanh cap and a distance bias.

A case is a dict of plain values; ``run`` computes it in plain torch operations
(``own`` false) or through the package's entry points (``own`` true).
"""

import math
import random

import torch

own = False


# ------------------------------------------------------------------ cases
def listed():
    return [
        # One decoding step of a small batch: every sequence gains one token.
        dict(name="append_tokens", op="append", dtype="bf16", hq=32, hkv=8, d=128, page=16,
             seqs=16, lo=1, hi=1, before=8000, rotary=128, interleaved=False, keep=False, mix=1),
        # The generation blocks of two long sequences (64 positions each), heads not shared.
        dict(name="append_blocks", op="append", dtype="bf16", hq=32, hkv=32, d=128, page=64,
             seqs=2, lo=64, hi=64, before=131072, rotary=128, interleaved=False, keep=False, mix=2),
        # A batch of ragged prompts entering the cache; rotated keys kept for the prefill.
        dict(name="append_prompts", op="append", dtype="bf16", hq=32, hkv=8, d=128, page=64,
             seqs=24, lo=3, hi=4096, before=0, rotary=128, interleaved=False, keep=True, mix=3),
        # Single precision, partial rotation of neighbouring pairs, an odd prompt length.
        dict(name="append_f32", op="append", dtype="f32", hq=2, hkv=2, d=64, page=32,
             seqs=1, lo=1021, hi=1021, before=17, rotary=32, interleaved=True, keep=True, mix=4),
        # One token for each of a few short conversations: latency counts.
        dict(name="token_short", op="paged", dtype="bf16", hq=32, hkv=8, d=128, page=16,
             seqs=4, lo=100, hi=1500, new=1, causal=True, prefix=False, cap=0.0, bias=False,
             idle=0, mix=5),
        # A serving batch of ragged lengths, two slots idle.
        dict(name="token_batch", op="paged", dtype="bf16", hq=32, hkv=8, d=128, page=16,
             seqs=64, lo=200, hi=16384, new=1, causal=True, prefix=False, cap=0.0, bias=False,
             idle=2, mix=6),
        # One token of one very long context, scores capped.
        dict(name="token_long", op="paged", dtype="bf16", hq=32, hkv=8, d=128, page=64,
             seqs=1, lo=131072, hi=131072, new=1, causal=True, prefix=False, cap=30.0, bias=False,
             idle=0, mix=7),
        # The 32-position generation block of a denoising step over two full caches.
        dict(name="block_long", op="paged", dtype="bf16", hq=32, hkv=32, d=128, page=64,
             seqs=2, lo=65536, hi=65536, new=32, causal=False, prefix=False, cap=0.0, bias=False,
             idle=0, mix=8),
        # The small single-precision layer's generation block.
        dict(name="block_f32", op="paged", dtype="f32", hq=2, hkv=2, d=64, page=32,
             seqs=1, lo=1056, hi=1056, new=32, causal=False, prefix=False, cap=0.0, bias=False,
             idle=0, mix=9),
        # The first denoising step's full attention over prompt and generation block.
        dict(name="prompt_full", op="prefill", dtype="bf16", hq=32, hkv=32, d=128,
             seqs=1, lo=4128, hi=4128, causal=False, prefix=False, cap=0.0, bias=False, mix=10),
        # Packed prompts of ragged lengths, causal after a bidirectional prefix each.
        dict(name="prompts_packed", op="prefill", dtype="bf16", hq=32, hkv=8, d=128,
             seqs=24, lo=20, hi=3000, causal=True, prefix=True, cap=0.0, bias=False, mix=11),
        # One long causal prompt with capped scores and a distance bias.
        dict(name="prompt_capped", op="prefill", dtype="bf16", hq=32, hkv=8, d=128,
             seqs=1, lo=16384, hi=16384, causal=True, prefix=False, cap=30.0, bias=True, mix=12),
    ]


def _spread(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    heads = [(32, 32), (32, 8), (16, 2), (8, 1), (2, 2), (12, 4), (5, 5), (9, 3)]
    hq, hkv = rng.choice(heads)
    case = dict(op=rng.choice(["append", "paged", "prefill"]),
                dtype="f32" if rng.random() < 0.2 else "bf16", hq=hq, hkv=hkv,
                d=rng.choice([64, 128, 128]), mix=rng.randrange(1 << 30))
    if case["op"] == "append":
        hi = _spread(rng, 1, 2048)
        rotary = rng.choice([case["d"], case["d"], case["d"] // 2, 16])
        case.update(page=rng.choice([8, 16, 32, 64, 128, 256]), seqs=_spread(rng, 1, 32),
                    lo=_spread(rng, 1, hi), hi=hi, before=_spread(rng, 1, 16384), rotary=rotary,
                    interleaved=rng.random() < 0.4, keep=rng.random() < 0.5)
        return case
    case.update(causal=rng.random() < 0.6, prefix=rng.random() < 0.3,
                cap=rng.choice([0.0, 0.0, 20.0, 50.0]), bias=rng.random() < 0.3)
    if case["op"] == "paged":
        new = rng.choice([1, 1, 1, 2, 5, 32, 64])
        seqs = _spread(rng, 1, 96)
        top = 131072 // seqs // (8 if case["dtype"] == "f32" else 1)
        hi = _spread(rng, max(new, 64), max(top, 128))
        case.update(page=rng.choice([8, 16, 32, 64, 128, 256]), seqs=seqs, new=new,
                    lo=_spread(rng, new, hi), hi=hi, idle=rng.choice([0, 0, 1]) if seqs > 1 else 0)
        return case
    seqs = _spread(rng, 1, 32)
    top = int((8192 if case["dtype"] == "bf16" else 2048) / math.sqrt(seqs))
    hi = _spread(rng, 8, top)
    case.update(seqs=seqs, lo=_spread(rng, 1, hi), hi=hi)
    return case


def _lengths(case):
    """Rows (append, prefill) or cache lengths (paged) of the case's sequences."""
    rng = random.Random(case["mix"])
    out = [_spread(rng, case["lo"], case["hi"]) for _ in range(case["seqs"])]
    for i in rng.sample(range(case["seqs"]), case.get("idle", 0)):
        out[i] = 0
    return out


def _before(case):
    """Rows already in the cache of each sequence (append)."""
    rng = random.Random(case["mix"] + 1)
    if case["before"] == 0:
        return [0] * case["seqs"]
    return [_spread(rng, 1 + case["before"] // 80, case["before"]) for _ in range(case["seqs"])]


def _prefixes(case, lengths):
    rng = random.Random(case["mix"] + 2)
    return [rng.randint(0, max(0, n // 2)) for n in lengths]


def _visible(case, n_q, n_k, prefix):
    """(query, key) pairs that the masks leave of one sequence and head."""
    if not case["causal"]:
        return n_q * n_k
    total = 0
    for i in range(n_q):
        total += min(n_k, max(n_k - n_q + i + 1, prefix))
    return total


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    lengths = _lengths(case)
    if case["op"] == "append":
        rows = sum(lengths)
        heads = 2 * (hq + 2 * hkv) + (hkv if case["keep"] else 0)
        pairs = rows * (hq + hkv) * case["rotary"] // 2
        return {"bytes": rows * heads * d * e, "flops": 6 * pairs}
    prefixes = _prefixes(case, lengths) if case["prefix"] else [0] * len(lengths)
    if case["op"] == "paged":
        rows = case["seqs"] * case["new"]
        keys = sum(lengths)
        pairs = sum(_visible(case, case["new"], n, p) for n, p in zip(lengths, prefixes) if n)
    else:
        rows = keys = sum(lengths)
        pairs = sum(_visible(case, n, n, p) for n, p in zip(lengths, prefixes))
    return {"bytes": 2 * keys * hkv * d * e + 2 * rows * hq * d * e + rows * hq * 4,
            "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------------ inputs
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _direction(gen, case):
    """One unit direction per key-value head; queries lean towards it, and so do
    the keys of planted spans, so that some keys matter far more than others."""
    u = _randn(gen, case["hkv"], case["d"])
    return u / u.norm(dim=-1, keepdim=True)


def _queries(gen, case, rows, u):
    g = case["hq"] // case["hkv"]
    q = _randn(gen, rows, case["hkv"], g, case["d"]) + 3.0 * u[None, :, None, :]
    return q.view(rows, case["hq"], case["d"]).to(_dtype(case))


def _scales(gen, case):
    s = torch.rand((case["d"],), generator=gen, device="cuda")
    return torch.exp(math.log(0.5) + s * math.log(4.0))


def _offsets(lengths):
    out = [0]
    for n in lengths:
        out.append(out[-1] + n)
    return out


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _slopes(case):
    n = case["hq"]
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / n) for h in range(n)], dtype=torch.float32,
                        device="cuda")


def _table(case, seed, totals):
    """Pages of each sequence, in no order, in a pool with a few pages to spare."""
    page = case["page"]
    need = [-(-n // page) for n in totals]
    order = list(range(sum(need) + 3))
    random.Random(seed).shuffle(order)
    rows, at = [], 0
    for n in need:
        rows.append(order[at:at + n] + [0] * (max(max(need), 1) - n))
        at += n
    return rows, len(order)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    lengths = _lengths(case)
    hq, hkv, d, dt = case["hq"], case["hkv"], case["d"], _dtype(case)
    state = {"case": case, "lengths": lengths}
    u = _direction(gen, case)
    scale = _scales(gen, case)
    if case["op"] == "append":
        before = _before(case)
        rows = sum(lengths)
        table, pages = _table(case, seed, [a + b for a, b in zip(before, lengths)])
        # The projections' output of the new rows; queries, keys and values side by side.
        qkv = torch.empty((rows, hq + 2 * hkv, d), dtype=dt, device="cuda")
        qkv[:, :hq] = _queries(gen, case, rows, u)
        qkv[:, hq:hq + hkv] = (_randn(gen, rows, hkv, d) * scale).to(dt)
        qkv[:, hq + hkv:] = _randn(gen, rows, hkv, d).to(dt)
        state.update(q=qkv[:, :hq], k=qkv[:, hq:hq + hkv], v=qkv[:, hq + hkv:], before=before,
                     table=table, dev_table=_int32(table), cu=_int32(_offsets(lengths)),
                     dev_before=_int32(before))
        pool = (pages, hkv, case["page"], d)
        state["cache"] = {"K": torch.full(pool, 0.5, dtype=dt, device="cuda"),
                          "V": torch.full(pool, -0.5, dtype=dt, device="cuda")}
        if own:
            from wavelet_guided_sparse_gb300 import binding as wf
            state["inv_freq"] = wf.rope_inv_freq(case["rotary"])
        return state
    state["prefixes"] = _prefixes(case, lengths) if case["prefix"] else None
    state["slopes"] = _slopes(case) if case["bias"] else None
    state["dev_prefix"] = _int32(state["prefixes"]) if case["prefix"] else None
    if case["op"] == "paged":
        table, pages = _table(case, seed, lengths)
        pool = (pages, hkv, case["page"], d)
        k = torch.empty(pool, dtype=dt, device="cuda")
        v = torch.empty(pool, dtype=dt, device="cuda")
        step = max(1, (1 << 26) // (hkv * case["page"] * d))
        for a in range(0, pages, step):  # in pieces: the draws are wider than the cache
            n = min(step, pages - a)
            keys = _randn(gen, n, hkv, case["page"], d) * scale
            keys[::16] += 3.0 * u[None, :, None, :]
            k[a:a + n] = keys.to(dt)
            v[a:a + n] = _randn(gen, n, hkv, case["page"], d).to(dt)
        q = _queries(gen, case, case["seqs"] * case["new"], u)
        state.update(q=q.view(case["seqs"], case["new"], hq, d), cache={"K": k, "V": v},
                     table=table, dev_table=_int32(table), kv_len=_int32(lengths))
        if own:
            from wavelet_guided_sparse_gb300 import binding as wf
            state["ws"] = wf.alloc_paged_attn_workspace(state["q"], state["cache"],
                                                        state["dev_table"])
        return state
    rows = sum(lengths)
    k = _randn(gen, rows, hkv, d) * scale
    k[::16] += 3.0 * u[None]
    state.update(q=_queries(gen, case, rows, u), k=k.to(dt), v=_randn(gen, rows, hkv, d).to(dt),
                 cu=_int32(_offsets(lengths)))
    return state


# ------------------------------------------------------------------ plain forms
def _turns(case, positions, device):
    """Cosine and sine [rows, rotary / 2] of the rotation, angles in 64 bits."""
    r = case["rotary"]
    i = torch.arange(r // 2, dtype=torch.float64, device=device)
    freq = torch.pow(torch.tensor(10000.0, dtype=torch.float64, device=device), -2.0 * i / r)
    angle = positions.to(torch.float64)[:, None] * freq[None]
    return torch.cos(angle), torch.sin(angle)


def _rotated(case, x, cos, sin):
    """x [rows, heads, d] in 32 bits with its first `rotary` channels rotated."""
    r = case["rotary"]
    x = x.float()
    c, s = cos.float()[:, None], sin.float()[:, None]
    if case["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack((a * c - b * s, a * s + b * c), dim=-1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        turned = torch.cat((a * c - b * s, a * s + b * c), dim=-1)
    return torch.cat((turned, x[..., r:]), dim=-1)


def _places(state):
    """Cache position, page and row within the page of every new row."""
    case, device = state["case"], state["q"].device
    pos = torch.cat([torch.arange(b, b + n, device=device)
                     for b, n in zip(state["before"], state["lengths"])])
    seq = torch.repeat_interleave(torch.arange(case["seqs"], device=device),
                                  torch.tensor(state["lengths"], device=device))
    page = state["dev_table"].long()[seq, pos // case["page"]]
    return pos, page, pos % case["page"]


def _append_plain(state):
    case, dt = state["case"], _dtype(state["case"])
    pos, page, row = _places(state)
    cos, sin = _turns(case, pos, pos.device)
    q = _rotated(case, state["q"], cos, sin).to(dt)
    k = _rotated(case, state["k"], cos, sin).to(dt)
    state["cache"]["K"][page, :, row] = k
    state["cache"]["V"][page, :, row] = state["v"]
    out = {"Q": q, "cache_K": state["cache"]["K"], "cache_V": state["cache"]["V"]}
    if case["keep"]:
        out["K"] = k
    return out


def _attend_plain(case, q, k, v, prefix, slopes):
    """One sequence: q [n_q, hq, d] at the last n_q positions of k, v [hkv, n_k, d]
    (32 bits); output [n_q, hq, d] and lse [n_q, hq], blocked over the queries."""
    n_q, hq, d = q.shape
    hkv, n_k = k.shape[0], k.shape[1]
    g = hq // hkv
    out = torch.zeros((n_q, hq, d), dtype=torch.float32, device=q.device)
    lse = torch.full((n_q, hq), -math.inf, dtype=torch.float32, device=q.device)
    if n_k == 0 or n_q == 0:
        return out, lse
    step = max(1, (1 << 27) // (hq * n_k))
    keys = torch.arange(n_k, device=q.device)
    for a in range(0, n_q, step):
        b = min(n_q, a + step)
        rows = b - a
        qb = q[a:b].view(rows, hkv, g, d).permute(1, 2, 0, 3).reshape(hkv, g * rows, d).float()
        z = torch.matmul(qb, k.transpose(1, 2)) * (1.0 / math.sqrt(d))
        z = z.view(hq, rows, n_k)
        if case["cap"] > 0.0:
            z = case["cap"] * torch.tanh(z / case["cap"])
        pos = n_k - n_q + torch.arange(a, b, device=q.device)
        if slopes is not None:
            z = z - slopes[:, None, None] * (pos[:, None] - keys[None]).abs().float()
        if case["causal"]:
            seen = (keys[None] <= pos[:, None]) | (keys[None] < prefix)
            z = z.masked_fill(~seen, -math.inf)
        top = z.amax(dim=-1, keepdim=True)
        p = torch.exp(z - top)
        total = p.sum(dim=-1, keepdim=True)
        o = torch.matmul(p.view(hkv, g * rows, n_k), v).view(hq, rows, d) / total
        out[a:b] = o.permute(1, 0, 2)
        lse[a:b] = (top + torch.log(total)).squeeze(-1).t()
    return out, lse


def _gathered(state, s, dtype):
    """Keys and values [hkv, n, d] of one sequence's pages."""
    case, n = state["case"], state["lengths"][s]
    pages = state["dev_table"][s, :-(-n // case["page"])].long()
    out = []
    for name in ("K", "V"):
        x = state["cache"][name][pages].to(dtype).permute(1, 0, 2, 3)
        out.append(x.reshape(case["hkv"], -1, case["d"])[:, :n])
    return out


def _paged_plain(state):
    case = state["case"]
    outs, lses = [], []
    for s in range(case["seqs"]):
        k, v = _gathered(state, s, torch.float32)
        prefix = state["prefixes"][s] if case["prefix"] else 0
        o, lse = _attend_plain(case, state["q"][s], k, v, prefix, state["slopes"])
        outs.append(o)
        lses.append(lse)
    return torch.stack(outs).to(_dtype(case)), torch.stack(lses)


def _prefill_plain(state):
    case = state["case"]
    outs, lses, at = [], [], 0
    for s, n in enumerate(state["lengths"]):
        k = state["k"][at:at + n].float().transpose(0, 1)
        v = state["v"][at:at + n].float().transpose(0, 1)
        prefix = state["prefixes"][s] if case["prefix"] else 0
        o, lse = _attend_plain(case, state["q"][at:at + n], k, v, prefix, state["slopes"])
        outs.append(o)
        lses.append(lse)
        at += n
    return torch.cat(outs).to(_dtype(case)), torch.cat(lses)


# ------------------------------------------------------------------ one pass
def run(state):
    case = state["case"]
    if not own:
        if case["op"] == "append":
            return _append_plain(state)
        return _paged_plain(state) if case["op"] == "paged" else _prefill_plain(state)
    from wavelet_guided_sparse_gb300 import binding as wf
    if case["op"] == "append":
        new = wf.paged_append(state["k"], state["v"], state["cache"], state["dev_table"],
                              state["cu"], state["dev_before"], q=state["q"],
                              inv_freq=state["inv_freq"], interleaved=case["interleaved"],
                              keep_keys=case["keep"])
        out = {"Q": new["Q"], "cache_K": state["cache"]["K"], "cache_V": state["cache"]["V"]}
        if case["keep"]:
            out["K"] = new["K"]
        return out
    options = dict(causal=case["causal"], prefix=state["dev_prefix"], softcap=case["cap"],
                   slopes=state["slopes"], with_lse=True)
    if case["op"] == "paged":
        return wf.paged_attn(state["q"], state["cache"], state["dev_table"], state["kv_len"],
                             state["ws"], **options)
    return wf.prefill_attn(state["q"], state["k"], state["v"], state["cu"], **options)


# ------------------------------------------------------------------ 64 bits
def _exact_rotation(case, x, pos):
    """Rotation by complex multiplication, in 64 bits."""
    r, x = case["rotary"], x.double()
    j = torch.arange(r // 2, dtype=torch.float64, device=x.device)
    turn = pos.double()[:, None] * torch.exp(-math.log(10000.0) * 2.0 * j / r)[None]
    w = torch.polar(torch.ones_like(turn), turn)[:, None]
    out = x.clone()
    if case["interleaved"]:
        y = torch.complex(x[..., 0:r:2].contiguous(), x[..., 1:r:2].contiguous()) * w
        out[..., 0:r:2], out[..., 1:r:2] = y.real, y.imag
    else:
        h = r // 2
        y = torch.complex(x[..., :h].contiguous(), x[..., h:r].contiguous()) * w
        out[..., :h], out[..., h:r] = y.real, y.imag
    return out


def _exact_append(state):
    case = state["case"]
    k_pool, v_pool = (state["cache"][n].double() for n in ("K", "V"))
    qs, ks, at = [], [], 0
    for s, n in enumerate(state["lengths"]):
        pos = torch.arange(state["before"][s], state["before"][s] + n, device="cuda")
        qs.append(_exact_rotation(case, state["q"][at:at + n], pos))
        ks.append(_exact_rotation(case, state["k"][at:at + n], pos))
        pages = torch.tensor(state["table"][s], device="cuda")[pos // case["page"]]
        k_pool[pages, :, pos % case["page"]] = ks[-1]
        v_pool[pages, :, pos % case["page"]] = state["v"][at:at + n].double()
        at += n
    out = {"Q": torch.cat(qs), "cache_K": k_pool, "cache_V": v_pool}
    if case["keep"]:
        out["K"] = torch.cat(ks)
    return out


def _exact_head(case, q, k, v, first, prefix, slope):
    """One head in 64 bits: q [n_q, d] at positions first.., k and v [n_k, d]."""
    n_k = k.shape[0]
    o = torch.zeros((q.shape[0], q.shape[1]), dtype=torch.float64, device=q.device)
    lse = torch.full((q.shape[0],), -math.inf, dtype=torch.float64, device=q.device)
    j = torch.arange(n_k, device=q.device)
    for a in range(0, q.shape[0], 2048):
        rows = q[a:a + 2048]
        if n_k == 0:
            break
        z = rows @ k.t() / math.sqrt(q.shape[1])
        if case["cap"] > 0.0:
            z = torch.tanh(z / case["cap"]) * case["cap"]
        i = first + a + torch.arange(rows.shape[0], device=q.device)
        if slope is not None:
            z -= slope * (i[:, None] - j[None]).abs()
        if case["causal"]:
            hidden = (j[None] > i[:, None]) & (j[None] >= prefix)
            z[hidden] = -math.inf
        lse[a:a + 2048] = torch.logsumexp(z, dim=1)
        o[a:a + 2048] = torch.softmax(z, dim=1) @ v
    return o, lse


def exact(case, seed):
    if work(case)["flops"] > 6e12:
        return None
    state = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(state)
    g = case["hq"] // case["hkv"]
    outs, lses, at = [], [], 0
    for s, n in enumerate(state["lengths"]):
        if case["op"] == "paged":
            q = state["q"][s].double()
            k, v = _gathered(state, s, torch.float64)
            first = n - case["new"]
        else:
            q = state["q"][at:at + n].double()
            k = state["k"][at:at + n].double().transpose(0, 1)
            v = state["v"][at:at + n].double().transpose(0, 1)
            first, at = 0, at + n
        prefix = state["prefixes"][s] if case["prefix"] else 0
        o = torch.empty_like(q)
        lse = torch.empty(q.shape[:2], dtype=torch.float64, device=q.device)
        for h in range(case["hq"]):
            slope = None if state["slopes"] is None else state["slopes"][h].double()
            o[:, h], lse[:, h] = _exact_head(case, q[:, h], k[h // g], v[h // g], first, prefix,
                                             slope)
        outs.append(o)
        lses.append(lse)
    if case["op"] == "paged":
        return torch.stack(outs), torch.stack(lses)
    return torch.cat(outs), torch.cat(lses)

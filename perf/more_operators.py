"""Operators of a serving loop around the paged cache: drafted trees, sliding
windows, and the pages themselves.

Five operators:

* tree: attention of a tree of drafted tokens per sequence over a paged cache;
* window: attention of one new token (or one generation block) per sequence over
  a paged cache, with a sliding window and first tokens that stay visible;
* prompt: the same window over packed prompts' own keys and values;
* fork: sequences that share their parent's pages, or copy them, in every layer;
* keep: listed rows of each sequence moved together in every layer, the pages
  behind them given back.

A case is a dict of plain values; ``run`` computes it in plain torch operations
(``own`` false) or through the package's entry points (``own`` true).
"""

import math
import random

import torch

own = False

FOREVER = 2 ** 31 - 1


# ------------------------------------------------------------------ cases
def listed():
    return [
        # A few short conversations, eight drafted tokens each: latency counts.
        dict(name="tree_small", op="tree", dtype="bf16", hq=32, hkv=8, d=128, page=16, seqs=4,
             lo=100, hi=1500, nodes=8, cap=0.0, bias=False, mix=1),
        # A serving batch of ragged lengths with up to 26 drafted tokens a sequence.
        dict(name="tree_batch", op="tree", dtype="bf16", hq=32, hkv=8, d=128, page=16, seqs=16,
             lo=1000, hi=16384, nodes=26, cap=0.0, bias=False, mix=2),
        # Long contexts and the widest trees.
        dict(name="tree_wide", op="tree", dtype="bf16", hq=32, hkv=8, d=128, page=64, seqs=4,
             lo=32768, hi=32768, nodes=64, cap=0.0, bias=False, mix=3),
        # A serving batch of a model whose layers look back 4096 tokens.
        dict(name="window_tokens", op="window", dtype="bf16", hq=32, hkv=8, d=128, page=16,
             seqs=64, lo=200, hi=32768, new=1, window=4096, sinks=4, causal=True, cap=0.0,
             bias=False, mix=4),
        # A 32-position generation block of a denoising step, heads not shared.
        dict(name="window_block", op="window", dtype="bf16", hq=32, hkv=32, d=128, page=64,
             seqs=4, lo=65536, hi=65536, new=32, window=8192, sinks=64, causal=False, cap=0.0,
             bias=False, mix=5),
        # One long prompt.
        dict(name="prompt_long", op="prompt", dtype="bf16", hq=32, hkv=8, d=128, seqs=1,
             lo=32768, hi=32768, window=4096, sinks=4, causal=True, cap=0.0, bias=False, mix=6),
        # Packed prompts of ragged lengths and a short window.
        dict(name="prompts_packed", op="prompt", dtype="bf16", hq=32, hkv=8, d=128, seqs=24,
             lo=20, hi=8192, window=1024, sinks=16, causal=True, cap=0.0, bias=False, mix=7),
        # The small single-precision layer, both directions.
        dict(name="prompt_f32", op="prompt", dtype="f32", hq=2, hkv=2, d=64, seqs=1, lo=4001,
             hi=4001, window=256, sinks=4, causal=False, cap=0.0, bias=False, mix=8),
        # Eight prompts into four candidates each: shared pages, the last one copied.
        dict(name="fork_beams", op="fork", dtype="bf16", hkv=8, d=128, page=16, layers=8, seqs=8,
             lo=100, hi=4000, children=4, share=True, mix=9),
        # Whole copies, for callers that rewrite prompt rows.
        dict(name="fork_copies", op="fork", dtype="bf16", hkv=8, d=128, page=64, layers=4, seqs=4,
             lo=16000, hi=16384, children=1, share=False, mix=10),
        # The accepted path of each drafted tree.
        dict(name="keep_path", op="keep", dtype="bf16", hkv=8, d=128, page=16, layers=8, seqs=16,
             lo=1000, hi=8192, drafted=26, most=7, mix=11),
        # An eighth of the rows of long contexts stays.
        dict(name="keep_rows", op="keep", dtype="bf16", hkv=8, d=128, page=64, layers=4, seqs=4,
             lo=32768, hi=32768, drafted=0, most=4096, mix=12),
    ]


def _spread(rng, lo, hi):
    """A whole number spread over the logarithm of [lo, hi]."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["tree", "window", "prompt", "fork", "keep"])
    hq, hkv = rng.choice([(32, 32), (32, 8), (16, 2), (8, 1), (2, 2), (12, 4), (5, 5), (9, 3)])
    case = dict(op=op, dtype="f32" if rng.random() < 0.2 else "bf16", hkv=hkv,
                d=rng.choice([64, 128, 128]), mix=rng.randrange(1 << 30))
    slow = 8 if case["dtype"] == "f32" else 1
    if op in ("fork", "keep"):
        case.update(page=rng.choice([8, 16, 32, 64, 128, 256]), layers=_spread(rng, 1, 12),
                    seqs=_spread(rng, 1, 16))
        children = _spread(rng, 1, 6) if op == "fork" else 1
        hi = (1 << 21) // (case["layers"] * case["seqs"] * hkv * children * slow)
        hi = _spread(rng, 16, max(64, min(hi, 65536)))
        case.update(lo=_spread(rng, 1, hi), hi=hi)
        if op == "fork":
            case.update(children=children, share=rng.random() < 0.6)
        else:
            drafted = rng.choice([0, 0, 1, 5, 26, 64])
            case.update(drafted=drafted, most=_spread(rng, 1, drafted or hi))
        return case
    case.update(hq=hq, cap=rng.choice([0.0, 0.0, 20.0, 50.0]), bias=rng.random() < 0.3)
    if op == "tree":
        case.update(nodes=_spread(rng, 1, 64), seqs=_spread(rng, 1, 48))
        hi = _spread(rng, 64, max(128, min((1 << 20) // (hkv * case["seqs"] * slow), 131072)))
        case.update(page=rng.choice([8, 16, 32, 64, 128, 256]), lo=_spread(rng, 1, hi), hi=hi)
        return case
    case.update(window=_spread(rng, 1, 8192 if op == "window" else 4096),
                sinks=rng.choice([0, 1, 4, 4, 16, 100]), causal=rng.random() < 0.7)
    if op == "window":
        new, seqs = rng.choice([1, 1, 1, 2, 5, 32, 64]), _spread(rng, 1, 64)
        hi = _spread(rng, max(new, 64), max(131072 // seqs // slow, 128))
        case.update(page=rng.choice([8, 16, 32, 64, 128, 256]), new=new, seqs=seqs,
                    lo=_spread(rng, new, hi), hi=hi)
        return case
    seqs = _spread(rng, 1, 32)
    hi = _spread(rng, 8, int((16384 if slow == 1 else 2048) / math.sqrt(seqs)))
    case.update(seqs=seqs, lo=_spread(rng, 1, hi), hi=hi)
    return case


def _lengths(case):
    """Rows of the case's sequences, their drafted tokens not counted."""
    rng = random.Random(case["mix"])
    return [_spread(rng, case["lo"], case["hi"]) for _ in range(case["seqs"])]


def _trees(case):
    """Parents of each sequence's drafted tokens (-1: it follows the last cached
    token): mostly near ones, as a drafter's best candidates have."""
    rng = random.Random(case["mix"] + 3)
    out = []
    for _ in range(case["seqs"]):
        n = rng.randint((case["nodes"] + 1) // 2, case["nodes"])
        out.append([-1] + [i - 1 if rng.random() < 0.5 else rng.randint(-1, i - 1)
                           for i in range(1, n)])
    return out


def _kept(case, lengths):
    """First row that may move and the rows that stay behind it, ascending."""
    rng = random.Random(case["mix"] + 4)
    if case["drafted"]:
        counts = [rng.randint(0, min(case["most"], case["drafted"])) for _ in lengths]
        return list(lengths), [[n + i for i in sorted(rng.sample(range(case["drafted"]), c))]
                               for n, c in zip(lengths, counts)]
    return [0] * len(lengths), [sorted(rng.sample(range(n), min(case["most"], n)))
                                for n in lengths]


def _depths(parents):
    out = []
    for p in parents:
        out.append(0 if p < 0 else out[p] + 1)
    return out


def _window_pairs(case, n, first):
    """(query, key) pairs that the window leaves to rows first..n-1, and the
    number of keys that some of them sees."""
    w, sinks = case["window"], min(case["sinks"], n)
    pairs = 0
    for p in range(first, n):
        hi = p + 1 if case["causal"] else min(n, p + w)
        lo = max(0, p - w + 1)
        pairs += hi - lo + min(sinks, lo)
    lo = max(0, first - w + 1)
    return pairs, n - lo + min(sinks, lo)


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    row = case["hkv"] * case["d"] * e
    lengths = _lengths(case)
    if case["op"] == "fork":
        page = case["page"]
        copied = sum(n % page if case["share"] else n for n in lengths) * case["children"]
        entries = sum(-(-n // page) for n in lengths) * case["children"]
        return {"bytes": 4 * case["layers"] * copied * row + 8 * entries, "flops": 0}
    if case["op"] == "keep":
        moved = sum(len(k) for k in _kept(case, lengths)[1])
        return {"bytes": 4 * case["layers"] * moved * row + 4 * moved + 8 * case["seqs"],
                "flops": 0}
    hq, d = case["hq"], case["d"]
    if case["op"] == "tree":
        trees = _trees(case)
        keys = sum(n + len(t) for n, t in zip(lengths, trees))
        rows = case["seqs"] * case["nodes"]
        pairs = sum(n * len(t) + sum(_depths(t)) + len(t) for n, t in zip(lengths, trees))
    else:
        new = case.get("new")
        got = [_window_pairs(case, n, 0 if new is None else n - new) for n in lengths]
        pairs, keys = sum(x[0] for x in got), sum(x[1] for x in got)
        rows = sum(lengths) if new is None else case["seqs"] * new
    return {"bytes": 2 * keys * row + 2 * rows * hq * d * e + rows * hq * 4,
            "flops": 4 * d * hq * pairs}


# ------------------------------------------------------------------ inputs
def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)


def _direction(gen, case):
    """One unit direction per key-value head; queries lean towards it, and so do
    some keys, so that some keys matter far more than others."""
    u = _randn(gen, case["hkv"], case["d"])
    return u / u.norm(dim=-1, keepdim=True)


def _queries(gen, case, rows, u):
    g = case["hq"] // case["hkv"]
    q = _randn(gen, rows, case["hkv"], g, case["d"]) + 3.0 * u[None, :, None, :]
    return q.view(rows, case["hq"], case["d"]).to(_dtype(case))


def _scales(gen, case):
    s = torch.rand((case["d"],), generator=gen, device="cuda")
    return torch.exp(math.log(0.5) + s * math.log(4.0))


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _slopes(case):
    n = case["hq"]
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / n) for h in range(n)], dtype=torch.float32,
                        device="cuda")


def _table(case, seed, totals, rows, spare):
    """Pages of each sequence, in no order, in a pool with some to spare; entries
    without a page are -1."""
    need = [-(-n // case["page"]) for n in totals]
    order = list(range(sum(need) + spare))
    random.Random(seed).shuffle(order)
    table, at = [], 0
    for n in need:
        table.append(order[at:at + n] + [-1] * (max(max(need), 1) - n))
        at += n
    table += [[-1] * len(table[0])] * (rows - len(table))
    return table, len(order)


def _prepare_pages(case, seed, gen, lengths):
    """Pools of every layer in one tensor, page table and reference counts."""
    page = case["page"]
    state = {}
    if case["op"] == "fork":
        rows = case["seqs"] * (1 + case["children"])
        need = sum(1 if case["share"] else -(-n // page) for n in lengths) * case["children"]
        table, pages = _table(case, seed, lengths, rows, need + 5)
        src = [s for s in range(case["seqs"]) for _ in range(case["children"])]
        dst = list(range(case["seqs"], rows))
        first = [0] * rows
        end = [0] * case["seqs"] + [FOREVER] * (rows - case["seqs"])
        state.update(src=_int32(src), dst=_int32(dst), first=_int32(first), end=_int32(end),
                     kv_len=_int32(lengths + [0] * (rows - case["seqs"])),
                     share=None if case["share"] else _int32([0] * len(src)))
    else:
        totals = [n + case["drafted"] for n in lengths]
        start, keep = _kept(case, lengths)
        table, pages = _table(case, seed, totals, case["seqs"], 5)
        width = max(1, max(len(k) for k in keep))
        state.update(kv_len=_int32(totals), start=_int32(start),
                     n_keep=_int32([len(k) for k in keep]),
                     keep=_int32([k + [0] * (width - len(k)) for k in keep]))
    pools = torch.empty((case["layers"], 2, pages, case["hkv"], page, case["d"]),
                        dtype=_dtype(case), device="cuda")
    pools.normal_(generator=gen)
    refs = torch.zeros(pages, dtype=torch.int32)
    refs[torch.tensor([p for row in table for p in row if p >= 0], dtype=torch.long)] = 1
    state.update(pools=pools, refs=refs.cuda(), table=_int32(table),
                 caches=[{"K": p[0], "V": p[1]} for p in pools])
    return state


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    lengths = _lengths(case)
    if case["op"] in ("fork", "keep"):
        return dict(_prepare_pages(case, seed, gen, lengths), case=case)
    hq, hkv, d, dt = case["hq"], case["hkv"], case["d"], _dtype(case)
    u, scale = _direction(gen, case), _scales(gen, case)
    state = {"case": case, "slopes": _slopes(case) if case["bias"] else None}
    if case["op"] == "prompt":
        rows = sum(lengths)
        k = _randn(gen, rows, hkv, d) * scale
        k[::16] += 3.0 * u[None]
        cu = [0]
        for n in lengths:
            cu.append(cu[-1] + n)
        state.update(q=_queries(gen, case, rows, u), k=k.to(dt), v=_randn(gen, rows, hkv, d).to(dt),
                     cu=_int32(cu), lengths=lengths)
        return state
    if case["op"] == "tree":
        trees = _trees(case)
        lengths = [n + len(t) for n, t in zip(lengths, trees)]
        state.update(parents=_int32([t + [-1] * (case["nodes"] - len(t)) for t in trees]),
                     tree_len=_int32([len(t) for t in trees]))
    new = case["nodes"] if case["op"] == "tree" else case["new"]
    table, pages = _table(case, seed, lengths, case["seqs"], 3)
    k = torch.empty((pages, hkv, case["page"], d), dtype=dt, device="cuda")
    v = torch.empty_like(k)
    step = max(1, (1 << 26) // (hkv * case["page"] * d))
    for a in range(0, pages, step):  # in pieces: the draws are wider than the cache
        n = min(step, pages - a)
        keys = _randn(gen, n, hkv, case["page"], d) * scale
        keys[::16] += 3.0 * u[None, :, None, :]
        k[a:a + n] = keys.to(dt)
        v[a:a + n] = _randn(gen, n, hkv, case["page"], d).to(dt)
    q = _queries(gen, case, case["seqs"] * new, u)
    state.update(q=q.view(case["seqs"], new, hq, d), cache={"K": k, "V": v}, table=_int32(table),
                 kv_len=_int32(lengths), lengths=lengths)
    return state


# ------------------------------------------------------------------ plain forms
def _softmax_plain(case, q, k, v, seen, dist, slopes):
    """q [.., hq, n, d], k and v [.., hkv, m, d] in 32 bits, seen and dist [.., 1
    or hq, n, m]: output [.., hq, n, d] and lse [.., hq, n]."""
    hq, n, d = q.shape[-3:]
    hkv, m = k.shape[-3:-1]
    lead, g = q.shape[:-3], hq // hkv
    qg = q.reshape(*lead, hkv, g * n, d)
    z = torch.matmul(qg, k.transpose(-1, -2)).mul_(1.0 / math.sqrt(d)).view(*lead, hq, n, m)
    if case["cap"] > 0.0:
        z = z.div_(case["cap"]).tanh_().mul_(case["cap"])
    if slopes is not None:
        z = z - slopes[:, None, None] * dist.float()
    z = z.masked_fill_(~seen, -math.inf)
    top = z.amax(dim=-1, keepdim=True)
    p = torch.exp(z.sub_(torch.where(top == -math.inf, 0.0, top)))
    total = p.sum(dim=-1, keepdim=True)
    o = torch.matmul(p.view(*lead, hkv, g * n, m), v).view(*lead, hq, n, d)
    o = o / torch.where(total == 0.0, 1.0, total)
    return o, (top + torch.log(total)).squeeze(-1)


def _rows_of(case, cache, table, rows):
    """Cache rows [S, m] of each sequence as [S, hkv, m, d] in 32 bits (rows
    outside a sequence read page 0)."""
    page = table.long().clamp(min=0).gather(1, (rows // case["page"]).clamp(0, table.shape[1] - 1))
    return [cache[n][page, :, rows % case["page"]].float().transpose(1, 2) for n in ("K", "V")]


def _tree_plain(state):
    case, table = state["case"], state["table"]
    n, length = case["nodes"], state["kv_len"].long()
    parents, count = state["parents"].long(), state["tree_len"].long()
    base = (length - count)[:, None]
    node = torch.arange(n, device=length.device)
    # Closure of the parent relation: [S, n, n], true where the second is the
    # first or one of its ancestors.
    up = ((parents[:, :, None] == node) | (node[:, None] == node)).float()
    for _ in range(6):
        up = (torch.matmul(up, up) > 0).float()
    depth = up.sum(dim=-1) - 1
    # The cached keys, then the drafted ones.
    old = torch.arange(max(state["lengths"]), device=length.device)[None].expand(len(length), -1)
    k, v = _rows_of(case, state["cache"], table, torch.cat((old, base + node), dim=1))
    there = node < count[:, None]
    seen = torch.cat(((old < base)[:, None].expand(-1, n, -1),
                      (up > 0) & there[:, None]), dim=2) & there[:, :, None]
    dist = None
    if case["bias"]:
        at = torch.cat((old.float(), base + depth), dim=1)
        dist = ((base + depth)[:, :, None] - at[:, None]).abs()[:, None]
    o, lse = _softmax_plain(case, state["q"].float().transpose(1, 2), k, v, seen[:, None], dist,
                            state["slopes"])
    return o.transpose(1, 2).to(_dtype(case)), lse.transpose(1, 2)


def _near(case, p, j):
    """Which keys j the window leaves to queries at p (sinks not counted)."""
    seen = (p - j < case["window"]) & (j >= case["sinks"])
    return seen & (j <= p) if case["causal"] else seen & (j - p < case["window"])


def _window_plain(state):
    """The keys of the sinks, then those of the window of a sequence's queries."""
    case, new, length = state["case"], state["case"]["new"], state["kv_len"].long()
    longest = max(state["lengths"])
    p = (length - new)[:, None] + torch.arange(new, device=length.device)
    sinks = torch.arange(min(case["sinks"], longest), device=length.device)[None]
    reach = torch.arange(min(case["window"] + new - 1, longest), device=length.device)
    far = (length[:, None] - len(reach)).clamp(min=0) + reach
    rows = torch.cat((sinks.expand(len(length), -1), far), dim=1)
    k, v = _rows_of(case, state["cache"], state["table"], rows)
    first = (sinks[:, None] <= p[:, :, None]) if case["causal"] else \
        torch.ones_like(p, dtype=torch.bool)[:, :, None].expand(-1, -1, sinks.shape[1])
    seen = torch.cat((first, _near(case, p[:, :, None], far[:, None])), dim=2)
    seen = seen & (rows < length[:, None])[:, None]
    dist = (p[:, :, None] - rows[:, None]).abs()[:, None] if case["bias"] else None
    o, lse = _softmax_plain(case, state["q"].float().transpose(1, 2), k, v, seen[:, None], dist,
                            state["slopes"])
    return o.transpose(1, 2).to(_dtype(case)), lse.transpose(1, 2)


def _prompt_plain(state):
    """All prompts in blocks of rows, a quarter of the window or 64: a block's keys
    are the sinks of its prompt and the rows that its window reaches."""
    case, cu, rows = state["case"], state["cu"].long(), state["q"].shape[0]
    device, b = cu.device, max(64, case["window"] // 4)
    longest = max(state["lengths"])
    count = cu[1:] - cu[:-1]
    blocks = -(-count // b)
    total = sum(-(-n // b) for n in state["lengths"])
    seq = torch.repeat_interleave(torch.arange(len(count), device=device), blocks,
                                  output_size=total)
    start = (torch.arange(total, device=device) - (blocks.cumsum(0) - blocks)[seq]) * b
    p = start[:, None] + torch.arange(b, device=device)
    w = min(case["window"], longest)
    sinks = torch.arange(min(case["sinks"], longest), device=device)[None]
    reach = torch.arange(1 - w, b if case["causal"] else b + w - 1, device=device)
    j = torch.cat((sinks.expand(total, -1), start[:, None] + reach), dim=1)
    inside = (j >= 0) & (j < count[seq][:, None])
    at = (cu[seq][:, None] + j).clamp(0, rows - 1)
    near = _near(case, p[:, :, None], j[:, None])
    first = torch.arange(j.shape[1], device=device) < sinks.shape[1]
    early = first & (j[:, None] <= p[:, :, None]) if case["causal"] else first
    seen = (near & ~first | early) & inside[:, None]
    dist = (p[:, :, None] - j[:, None]).abs()[:, None] if case["bias"] else None
    k, v = (state[x][at].float().transpose(1, 2) for x in ("k", "v"))
    take = (cu[seq][:, None] + p).clamp(max=rows - 1)
    o, lse = _softmax_plain(case, state["q"][take].float().transpose(1, 2), k, v, seen[:, None],
                            dist, state["slopes"])
    there = p < count[seq][:, None]
    return (o.transpose(1, 2)[there].to(_dtype(case)), lse.transpose(1, 2)[there])


def _take_free(refs, wanted, table):
    """Entries of the table marked in `wanted`, in order, get the lowest free pages."""
    order = torch.argsort((refs != 0).to(torch.int8), stable=True)
    rank = (wanted.flatten().cumsum(0) - 1).clamp(0, len(refs) - 1).view(wanted.shape)
    page = order[rank].to(torch.int32)
    refs.scatter_add_(0, page.long().flatten(), wanted.flatten().to(torch.int32))
    return torch.where(wanted, page, table)


def _fork_plain(state):
    case, table, refs, pools = state["case"], state["table"], state["refs"], state["pools"]
    page, src, dst = case["page"], state["src"].long(), state["dst"].long()
    length = state["kv_len"].long()[src][:, None]
    entry = torch.arange(table.shape[1], device=table.device)[None]
    held = entry * page < length
    shared = (entry + 1) * page <= length if state["share"] is None else torch.zeros_like(held)
    parent = table[src]
    child = torch.where(held & shared, parent, -1)
    refs.scatter_add_(0, parent.long().clamp(min=0).flatten(),
                      (held & shared).flatten().to(torch.int32))
    child = _take_free(refs, held & ~shared, child)
    table[dst] = child
    # Rows of the copied pages, all layers, keys and values at once.
    row = torch.arange(page, device=table.device)
    copied = (held & ~shared)[:, :, None] & (entry[:, :, None] * page + row < length[:, :, None])
    fork, e, r = copied.nonzero(as_tuple=True)
    lines = pools.permute(0, 1, 3, 2, 4, 5)
    lines[:, :, :, child[fork, e].long(), r] = lines[:, :, :, parent[fork, e].long(), r]
    forked = table.clone()
    # The children have ended: their pages go back.
    begin, end = state["first"].long()[:, None], state["end"].long()[:, None]
    gone = (entry * page >= begin) & ((entry + 1) * page <= end) & (table >= 0)
    refs.scatter_add_(0, table.long().clamp(min=0).flatten(), -gone.flatten().to(torch.int32))
    table.masked_fill_(gone, -1)
    return {"table": forked, "refs": refs, "pools": pools}


def _keep_plain(state):
    case, table, refs, pools = state["case"], state["table"], state["refs"], state["pools"]
    page, length = case["page"], state["kv_len"].long()[:, None]
    entry = torch.arange(table.shape[1], device=table.device)[None]
    table.copy_(_take_free(refs, (entry * page < length) & (table < 0), table))
    keep, start, count = state["keep"].long(), state["start"].long(), state["n_keep"].long()
    i = torch.arange(keep.shape[1], device=table.device)[None]
    s, i = (i < count[:, None]).nonzero(as_tuple=True)
    old, new = keep[s, i], start[s] + i
    lines = pools.permute(0, 1, 3, 2, 4, 5)
    moved = lines[:, :, :, table[s, old // page].long(), old % page]
    lines[:, :, :, table[s, new // page].long(), new % page] = moved
    gone = (entry * page >= (start + count)[:, None]) & (table >= 0)
    refs.scatter_add_(0, table.long().clamp(min=0).flatten(), -gone.flatten().to(torch.int32))
    table.masked_fill_(gone, -1)
    return {"table": table, "refs": refs, "pools": pools}


# ------------------------------------------------------------------ one pass
def _run_own(state):
    from wavelet_guided_sparse_gb300 import binding as wf
    case = state["case"]
    if case["op"] == "fork":
        if "ws" not in state:  # what a program keeps: its layers' handle, a workspace
            state["layers"] = wf.page_pools(state["caches"])
            state["ws"] = wf.alloc_pages_workspace(state["layers"], state["table"],
                                                   max_forks=len(state["src"]))
        call = dict(refs=state["refs"], ws=state["ws"])
        wf.paged_fork(state["layers"], state["table"], src=state["src"], dst=state["dst"],
                      kv_len=state["kv_len"], share_rows=state["share"], **call)
        forked = state["table"].clone()
        wf.paged_release(state["layers"], state["table"], first=state["first"],
                         end=state["end"], **call)
        return {"table": forked, "refs": state["refs"], "pools": state["pools"]}
    if case["op"] == "keep":
        if "ws" not in state:
            state["layers"] = wf.page_pools(state["caches"])
            state["ws"] = wf.alloc_pages_workspace(state["layers"], state["table"],
                                                   max_keep=state["keep"].shape[1])
        call = dict(refs=state["refs"], ws=state["ws"])
        wf.paged_reserve(state["layers"], state["table"], rows=state["kv_len"], **call)
        wf.paged_keep(state["layers"], state["table"], kv_len=state["kv_len"],
                      start=state["start"], keep=state["keep"], n_keep=state["n_keep"], **call)
        return {"table": state["table"], "refs": state["refs"], "pools": state["pools"]}
    options = dict(softcap=case["cap"], slopes=state["slopes"], with_lse=True)
    if case["op"] == "tree":
        if "ws" not in state:
            state["ws"] = wf.alloc_paged_tree_workspace(state["q"], state["cache"], state["table"])
        return wf.paged_tree_attn(state["q"], state["cache"], state["table"], state["kv_len"],
                                  state["parents"], state["ws"], tree_len=state["tree_len"],
                                  **options)
    options.update(window=case["window"], sinks=case["sinks"], causal=case["causal"])
    if case["op"] == "window":
        if "ws" not in state:
            state["ws"] = wf.alloc_paged_attn_workspace(state["q"], state["cache"], state["table"])
        return wf.paged_window_attn(state["q"], state["cache"], state["table"], state["kv_len"],
                                    ws=state["ws"], **options)
    return wf.prefill_window_attn(state["q"], state["k"], state["v"], state["cu"], **options)


def run(state):
    if own:
        return _run_own(state)
    return {"tree": _tree_plain, "window": _window_plain, "prompt": _prompt_plain,
            "fork": _fork_plain, "keep": _keep_plain}[state["case"]["op"]](state)


# ------------------------------------------------------------------ 64 bits
def _exact_rows(case, q, k, v, p, at, seen, slope):
    """One head in 64 bits: q [n, d] at positions p, keys k [m, d] at positions at."""
    z = q @ k.t() / math.sqrt(q.shape[1])
    if case["cap"] > 0.0:
        z = torch.tanh(z / case["cap"]) * case["cap"]
    if slope is not None:
        z -= slope * (p[:, None] - at[None]).abs()
    z[~seen] = -math.inf
    lse = torch.logsumexp(z, dim=1)
    o = torch.softmax(z, dim=1).nan_to_num(0.0) @ v
    return o, lse


def _exact_attention(case, state, s):
    """One sequence: (queries' positions, output, lse) rows, head by head."""
    hq, g, page = case["hq"], case["hq"] // case["hkv"], case.get("page")
    n = state["lengths"][s]
    if case["op"] == "prompt":
        a = int(state["cu"][s])
        q, k, v = (state[x][a:a + n].double() for x in ("q", "k", "v"))
        p = torch.arange(n, device="cuda")
    else:
        q = state["q"][s].double()
        pages = state["table"][s, :-(-n // page)].long()
        k, v = (state["cache"][x][pages].double().transpose(1, 2).flatten(0, 1)[:n]
                for x in ("K", "V"))
        p = n - q.shape[0] + torch.arange(q.shape[0], device="cuda")
    at = torch.arange(n, device="cuda")
    o = torch.zeros_like(q)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    if case["op"] == "tree":
        count = int(state["tree_len"][s])
        tree = state["parents"][s, :count].tolist()
        base, depth = n - count, _depths(tree)
        seen = torch.zeros((count, n), dtype=torch.bool)
        for i in range(count):
            seen[i, :base] = True
            a = i
            while a >= 0:
                seen[i, base + a] = True
                a = tree[a]
        p = base + torch.tensor(depth, device="cuda")
        at[base:] = p
        spans = [(0, count, 0, n, seen.cuda())]
    else:
        spans = []
        for a in range(0, len(p), 1024):
            b = min(len(p), a + 1024)
            lo = max(0, int(p[a]) - case["window"] + 1)
            hi = n if not case["causal"] else int(p[b - 1]) + 1
            hi = min(n, hi, int(p[b - 1]) + case["window"])
            spans.append((a, b, lo, hi, None))
    for a, b, lo, hi, seen in spans:
        cols = at.new_tensor(range(0)) if seen is not None else \
            torch.arange(min(case["sinks"], lo, n), device="cuda")
        cols = torch.cat((cols, torch.arange(lo, hi, device="cuda")))
        if seen is None:
            away = p[a:b, None] - cols[None]
            seen = (away < case["window"]) | (cols[None] < case["sinks"])
            seen &= (away >= 0) if case["causal"] else \
                ((-away < case["window"]) | (cols[None] < case["sinks"]))
        for h in range(hq):
            slope = None if state["slopes"] is None else state["slopes"][h].double()
            o[a:b, h], lse[a:b, h] = _exact_rows(case, q[a:b, h], k[cols, h // g], v[cols, h // g],
                                                 p[a:b], at[cols], seen, slope)
    return o, lse


def _exact_pages(case, state):
    """The pages' bookkeeping entry by entry, rows copied one page at a time."""
    page = case["page"]
    table, refs = state["table"].tolist(), state["refs"].tolist()
    pools = state["pools"].double()

    def take():
        p = refs.index(0)
        refs[p] = 1
        return p

    def drop(s, gone):
        for e, p in enumerate(table[s]):
            if p >= 0 and gone(e):
                refs[p] -= 1
                table[s][e] = -1

    if case["op"] == "fork":
        copies = []
        for a, b in zip(state["src"].tolist(), state["dst"].tolist()):
            n = int(state["kv_len"][a])
            full = n // page if case["share"] else 0
            for e in range(full):
                table[b][e] = table[a][e]
                refs[table[a][e]] += 1
            copies += [(a, b, e, min(page, n - e * page)) for e in range(full, -(-n // page))]
        for a, b, e, rows in copies:
            table[b][e] = take()
            pools[:, :, table[b][e], :, :rows] = pools[:, :, table[a][e], :, :rows]
        forked = [list(row) for row in table]
        for s in range(case["seqs"], len(table)):
            drop(s, lambda e: True)
    else:
        for s, n in enumerate(state["kv_len"].tolist()):
            for e in range(-(-n // page)):
                if table[s][e] < 0:
                    table[s][e] = take()
        start, count = state["start"].tolist(), state["n_keep"].tolist()
        for s, old in enumerate(state["keep"].tolist()):
            old = old[:count[s]]
            new = range(start[s], start[s] + len(old))
            rows = pools[:, :, [table[s][i // page] for i in old], :, [i % page for i in old]]
            pools[:, :, [table[s][i // page] for i in new], :, [i % page for i in new]] = rows
            drop(s, lambda e: e * page >= start[s] + len(old))
        forked = table
    return {"table": _int32(forked), "refs": _int32(refs), "pools": pools}


def exact(case, seed):
    if case["op"] in ("fork", "keep"):
        return _exact_pages(case, prepare(case, seed))
    if work(case)["flops"] > 4e12:
        return None
    state = prepare(case, seed)
    outs = []
    for s in range(case["seqs"]):
        if case["op"] == "tree":  # rows without a node: nothing visible
            n, live = case["nodes"], int(state["tree_len"][s])
            sub = dict(state, q=state["q"][:, :live])
            o, lse = _exact_attention(case, sub, s)
            o = torch.cat((o, o.new_zeros((n - live, *o.shape[1:]))))
            lse = torch.cat((lse, lse.new_full((n - live, lse.shape[1]), -math.inf)))
        else:
            o, lse = _exact_attention(case, state, s)
        outs.append((o, lse))
    join = torch.cat if case["op"] == "prompt" else torch.stack
    return join([o for o, _ in outs]), join([x for _, x in outs])

"""Cases of the operators around the paged K/V cache: norms and rotation of queries
and keys in front of it, forking and compacting its pages, and attention over the
blocks that a cheap score selects.

Each operator has a plain form (elementary torch operations in 32 bits; angles in
64) and the framework's own call; ``own`` says which one ``run`` makes.  ``exact``
gives the operators' definitions in 64 bits.
"""
from __future__ import annotations

import math
import random

import torch

own = False


# ------------------------------------------------------------------ cases

def _rotate(dim, heads, kv_heads, rows, axes, style, pairing, norm, far, name=None):
    return _named({"op": "rotate", "dim": dim, "heads": heads, "kv_heads": kv_heads, "rows": rows, "axes": axes,
                   "style": style, "pairing": pairing, "norm": norm, "far": far}, name)


def _pages(op, kind, dim, kv_heads, page, n, children, lo, hi, share, mix, name=None):
    """fork: n parents of lo .. hi tokens, `children` each.  compact: n sequences, whose
    pages fill `share` of the pool."""
    return _named({"op": op, "kind": kind, "dim": dim, "kv_heads": kv_heads, "page": page, "n": n,
                   "children": children, "lo": lo, "hi": hi, "share": share, "mix": mix}, name)


def _sparse(op, kind, dim, heads, kv_heads, page, n, chunk, history, top, first, last, mix, name=None):
    return _named({"op": op, "kind": kind, "dim": dim, "heads": heads, "kv_heads": kv_heads, "page": page, "n": n,
                   "chunk_lo": chunk[0], "chunk_hi": chunk[1], "hist_lo": history[0], "hist_hi": history[1],
                   "top": top, "first": first, "last": last, "mix": mix}, name)


def _named(c, name):
    if name is not None:
        c["name"] = name
    return c


def listed():
    return [
        # One new token of each of 48 running sequences, three position axes: all latency.
        _rotate(128, 40, 8, 48, 3, "interleaved", "half_vector", True, 30000, name="rotate_step"),
        # The rows of a prefill chunk of several prompts, positions far into a long context.
        _rotate(128, 40, 8, 8500, 3, "sections", "half_vector", True, 1000000, name="rotate_chunk"),
        # A step of a beam search: 16 prompts, the 4 beams of each start again from one sequence.
        _pages("fork", "bf16", 128, 8, 16, 16, 4, 500, 6000, 1.0, 1, name="fork_beams_bf16"),
        # Many samples of a few long prompts, quantised, larger pages.
        _pages("fork", "e4m3", 128, 8, 64, 6, 40, 8000, 40000, 1.0, 2, name="fork_samples_e4m3"),
        # A small pool after a few sequences have left.
        _pages("compact", "bf16", 64, 4, 32, 12, 0, 100, 3000, 0.5, 3, name="compact_small_bf16"),
        # A pool of 1 GB, two thirds full, whose free end is wanted back.
        _pages("compact", "bf16", 128, 8, 64, 40, 0, 1000, 9000, 0.65, 4, name="compact_large_bf16"),
        # One new token of each of 64 sequences: a page is completed now and then.
        _sparse("bounds", "bf16", 128, 40, 8, 16, 64, (1, 1), (500, 8000), 64, 1, 2, 5, name="bounds_step_bf16"),
        # The pages that the chunks of three long prompts completed.
        _sparse("bounds", "e4m3", 128, 40, 8, 64, 3, (2000, 6000), (0, 9000), 64, 1, 2, 6, name="bounds_chunk_e4m3"),
        # Selection for one new token of each of 48 long sequences.
        _sparse("select", "bf16", 128, 40, 8, 64, 48, (1, 1), (8000, 60000), 64, 1, 2, 7, name="select_step_bf16"),
        # Selection for every row of a chunk of a long prompt.
        _sparse("select", "bf16", 128, 40, 8, 64, 1, (2048, 2048), (32000, 32000), 16, 1, 2, 8,
                name="select_chunk_bf16"),
        # Attention of one new token of each of 48 long sequences over 64 blocks of 64 tokens.
        _sparse("attend", "bf16", 128, 40, 8, 64, 48, (1, 1), (8000, 60000), 64, 1, 2, 9, name="attend_step_bf16"),
        # Attention of the rows of a chunk of a long prompt over 16 blocks each, quantised pages: the largest.
        _sparse("attend", "e4m3", 128, 40, 8, 64, 1, (2048, 2048), (32000, 32000), 16, 1, 2, 10,
                name="attend_chunk_e4m3"),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the same ranges, no dearer than the largest listed."""
    most = max(w["bytes"] + w["flops"] / 280 for w in map(work, listed()))
    while True:
        op = rng.choice(["rotate", "fork", "compact", "bounds", "select", "attend", "attend"])
        kind = rng.choice(["bf16", "e4m3"])
        dim = rng.choice([64, 128])
        kv_heads = rng.choice([1, 2, 4, 8, 8, 10])
        heads = kv_heads * rng.choice([1, 2, 4, 5, 7, 8, 16])
        page = rng.choice([16, 32, 64, 128])
        mix = rng.randrange(1, 1 << 30)
        if op == "rotate":
            axes = rng.choice([1, 3])
            style = rng.choice(["interleaved", "sections"]) if axes == 3 else "one"
            c = _rotate(dim, heads, kv_heads, _log_uniform(rng, 1, 20000), axes, style,
                        rng.choice(["half_vector", "adjacent"]), rng.random() < 0.8, _log_uniform(rng, 100, 1000000))
        elif op in ("fork", "compact"):
            lo = _log_uniform(rng, 1, 20000)
            c = _pages(op, kind, dim, kv_heads, page, _log_uniform(rng, 1, 60),
                       _log_uniform(rng, 1, 40) if op == "fork" else 0, lo, _log_uniform(rng, lo, 40000),
                       1.0 if op == "fork" else rng.uniform(0.2, 0.95), mix)
        else:
            lo = _log_uniform(rng, 1, 2500)
            chunk = rng.choice([(1, 1), (1, 8), (lo, _log_uniform(rng, lo, 2500))])
            hist = _log_uniform(rng, 100, 60000)
            n = _log_uniform(rng, 1, 64) if chunk[1] <= 8 else _log_uniform(rng, 1, 4)
            first, last = rng.choice([0, 1, 1, 4]), rng.choice([1, 1, 2, 5])
            top = max(first + last, _log_uniform(rng, 4, 4096 // page))
            c = _sparse(op, kind, dim, heads, kv_heads, page, n, chunk, (_log_uniform(rng, 1, hist), hist), top,
                        first, last, mix)
        w = work(c)
        # A call takes up to 1024 sequences; what the plain form gathers, and the inputs, stay within a few GB.
        if op == "fork" and c["n"] * c["children"] > 1024 or op == "bounds" and not w["flops"]:
            continue
        if w["bytes"] + w["flops"] / 280 <= most and _held(c) < 9e9:
            return c


def _held(case):
    """Bytes that the plain form and the inputs hold, roughly."""
    op, d = case["op"], case["dim"]
    if op == "rotate":
        return case["rows"] * (case["heads"] + 2 * case["kv_heads"]) * d * 16
    if op in ("fork", "compact"):
        tokens = sum(_lengths(case)) / case["share"] + case["n"] * (case["children"] + 1) * case["page"]
        return tokens * case["kv_heads"] * d * 4
    q, kv = _chunks(case)
    pool = sum(kv) * case["kv_heads"] * d * 24
    if op == "bounds":
        return pool
    scores = sum(q) * case["kv_heads"] * (max(kv) // case["page"] + 1) * 40
    seen = case["top"] * case["page"] if op == "attend" else 0
    return pool + scores + sum(q) * case["kv_heads"] * seen * (d * 8 + 4 * case["heads"] // case["kv_heads"])


def _between(r, lo, hi):
    return lo if lo == hi else _log_uniform(r, max(lo, 1), hi)


def _lengths(case):
    r = random.Random(case["mix"])
    return [_between(r, case["lo"], case["hi"]) for _ in range(case["n"])]


def _chunks(case):
    """New tokens and cached tokens (those included) of each sequence."""
    r = random.Random(case["mix"])
    q = [_between(r, case["chunk_lo"], case["chunk_hi"]) for _ in range(case["n"])]
    return q, [c + _between(r, case["hist_lo"], case["hist_hi"]) if case["hist_hi"] else c for c in q]


def _pool_of(case):
    """(pages that the sequences use, pages of the pool) of a compaction."""
    used = [-(-x // case["page"]) for x in _lengths(case)]
    used = sum(u - _shared(used, s) for s, u in enumerate(used))
    return used, max(used + 1, int(used / case["share"]))


def _shared(used, s):
    """Every other sequence of a pool shares the first half of what its neighbour has."""
    return min(used[s], used[s - 1]) // 2 if s % 2 else 0


def work(case):
    op, d, hk, page = case["op"], case["dim"], case["kv_heads"], case.get("page", 1)
    if op == "rotate":
        n = case["rows"] * (case["heads"] + hk) * d
        return {"bytes": 4 * n + 4 * case["axes"] * case["rows"], "flops": 8 * n}
    held = 2 * d if case["kind"] == "bf16" else d + 1      # bytes of one key or value
    if op == "fork":
        kv = _lengths(case)
        entries = sum(x // page for x in kv) * case["children"]
        copies = sum(x % page != 0 for x in kv) * case["children"]
        # A table entry is read and written; a count of each shared page is read and written.
        return {"bytes": 8 * entries + 8 * sum(x // page for x in kv) + copies * page * hk * 4 * held, "flops": 0}
    if op == "compact":
        used, pool = _pool_of(case)
        moved = used * (pool - used) / pool
        return {"bytes": moved * page * hk * 4 * held + 8 * used + 8 * pool, "flops": 0}
    q, kv = _chunks(case)
    if op == "bounds":
        done = sum(l // page - (l - c) // page for c, l in zip(q, kv))
        return {"bytes": done * hk * (page * held + 2 * d + 1) + 4 * done + 8 * len(kv),
                "flops": 2 * done * hk * page * d}
    g = case["heads"] // hk
    if op == "select":
        blocks = sum(l // page for l in kv)
        pairs = sum(c * (l // page) for c, l in zip(q, kv))
        return {"bytes": blocks * hk * (2 * d + 1) + sum(q) * (case["heads"] * d * 2 + hk * case["top"] * 4),
                "flops": 4.0 * pairs * hk * d}
    read = pairs = 0
    for c, l in zip(q, kv):
        read += min(l, c * case["top"] * page)
        pairs += c * min(l, case["top"] * page)
    return {"bytes": sum(q) * (case["heads"] * d * 4 + hk * case["top"] * 4) + read * hk * 2 * held,
            "flops": 4.0 * pairs * hk * g * d}


# ------------------------------------------------------------------ inputs

def _quantise(x):
    """bf16 rows [..., d] -> (e4m3 bits of x 2^-e, exponent bytes e + 127): 448 2^e covers the row."""
    frac, ex = torch.frexp(x.float().abs().amax(-1))
    e = torch.where(frac <= 0.875, ex - 9, ex - 8).clamp_min(-117)
    bits = torch.ldexp(x.float(), -e.unsqueeze(-1)).to(torch.float8_e4m3fn).view(torch.uint8)
    return bits, (e + 127).to(torch.uint8)


def _fill_pages(state, case, n_pages, gen, parts=("k", "v")):
    """Keys or values as a projection leaves them: unequal channels, a few large ones."""
    hk, d = case["kv_heads"], case["dim"]
    channel = torch.exp(0.4 * torch.randn((hk, 1, d), generator=gen, device="cuda"))
    state["n_pages"] = n_pages
    for x in parts:
        held = torch.randn((n_pages, hk, case["page"], d), generator=gen, device="cuda", dtype=torch.float32)
        held = held.mul_(channel).to(torch.bfloat16)
        state[x + "_exp"] = None
        if case["kind"] == "e4m3":
            held, state[x + "_exp"] = _quantise(held)
        state[x] = held


def _int(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _prepare_rotate(state, case, gen):
    rows, d, hq, hk = case["rows"], case["dim"], case["heads"], case["kv_heads"]
    state["qkv"] = torch.randn((rows, (hq + 2 * hk) * d), generator=gen, device="cuda").to(torch.bfloat16)
    # Positions as chunks of prompts have them: text on a line, images spread over their axes.
    start = torch.randint(0, case["far"], (rows,), generator=gen, device="cuda")
    state["positions"] = torch.stack([start + torch.randint(0, 64, (rows,), generator=gen, device="cuda")
                                      for _ in range(case["axes"])]).to(torch.int32)
    state["q_norm"] = state["k_norm"] = None
    if case["norm"]:
        state["q_norm"], state["k_norm"] = ((1 + 0.1 * torch.randn((d,), generator=gen, device="cuda")).to(
            torch.bfloat16) for _ in range(2))
    state["q_out"] = torch.zeros((rows, hq, d), dtype=torch.bfloat16, device="cuda")
    state["k_out"] = torch.zeros((rows, hk, d), dtype=torch.bfloat16, device="cuda")


def _prepare_pages(state, case, gen):
    kv, page, kids = _lengths(case), case["page"], case["children"]
    used = [-(-x // page) for x in kv]
    n, cols = case["n"], max(used) + 1
    slots = n * (1 + kids)
    n_pages = sum(used) + n * kids + 3 if case["op"] == "fork" else _pool_of(case)[1]
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((slots, cols), -1, dtype=torch.int32, device="cuda")
    at = 0
    for s, u in enumerate(used):
        shared = _shared(used, s) if case["op"] == "compact" else 0
        table[s, :shared] = table[s - 1, :shared]
        table[s, shared:u] = order[at:at + u - shared]
        at += u - shared
    live = table[table >= 0].long()
    state.update(table=table, kv_len=_int(kv + [0] * (n * kids)), refs=torch.bincount(live, minlength=n_pages).int())
    _fill_pages(state, case, n_pages, gen)
    if case["op"] == "fork":
        state["src"] = torch.arange(n, device="cuda").repeat_interleave(kids).to(torch.int32)
        state["dst"] = torch.arange(n, n + n * kids, device="cuda").to(torch.int32)
        state["none"] = torch.zeros_like(state["dst"])
    else:
        state["was"] = tuple(state[x].clone() for x in ("table", "refs"))


def _prepare_sparse(state, case, gen):
    q, kv = _chunks(case)
    n, d, hk, hq, page = case["n"], case["dim"], case["kv_heads"], case["heads"], case["page"]
    rows, used = sum(q), [-(-l // page) for l in kv]
    order = torch.randperm(sum(used) + 3, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((n, max(used)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for s, u in enumerate(used):
        table[s, :u] = order[at:at + u]
        at += u
    state.update(rows=rows, max_rows=max(q), table=table, kv_len=_int(kv),
                 row_off=_int([sum(q[:i]) for i in range(n + 1)]))
    _fill_pages(state, case, len(order), gen, ("k", "v") if case["op"] == "attend" else ("k",))
    shape = (len(order), hk, 2, d)
    if case["op"] == "bounds":
        state["bounds"] = torch.zeros(shape, dtype=torch.int8, device="cuda")
        state["bounds_exp"] = torch.full(shape[:2], 127, dtype=torch.uint8, device="cuda")
        state["v"], state["v_exp"] = state["k"], state["k_exp"]      # values have no part in it
        return
    whole = torch.arange(len(order), device="cuda")
    state["bounds"], state["bounds_exp"] = _bounds_of(_values(state["k"], state["k_exp"], whole))
    state["qkv"] = torch.randn((rows, (hq + 2 * hk) * d), generator=gen, device="cuda").to(torch.bfloat16)
    if case["op"] == "select":
        state["v"], state["v_exp"] = state["k"], state["k_exp"]
        state["blocks"] = torch.full((rows, hk, case["top"]), -1, dtype=torch.int32, device="cuda")
    else:
        state["blocks"] = _plain_select(state)
        state["out"] = torch.zeros((rows, hq, d), dtype=torch.bfloat16, device="cuda")


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    state = {"case": case, "status": torch.zeros(1, dtype=torch.int32, device="cuda")}
    if case["op"] == "rotate":
        _prepare_rotate(state, case, gen)
    elif case["op"] in ("fork", "compact"):
        _prepare_pages(state, case, gen)
    else:
        _prepare_sparse(state, case, gen)
    return state


# ------------------------------------------------------------------ plain forms

THETA, EPS = 1000000.0, 1e-6


def _sections(case):
    """Pairs of a head on each axis (the first one has the rest)."""
    pairs = case["dim"] // 2
    side = (pairs * 5) // 16
    return (pairs - 2 * side, side, side) if case["axes"] == 3 else (pairs,)


def _axis_of_pair(case):
    i = torch.arange(case["dim"] // 2)
    if case["axes"] == 1:
        return torch.zeros_like(i)
    s = _sections(case)
    if case["style"] == "sections":
        return (i >= s[0]).long() + (i >= s[0] + s[1]).long()
    a = i % 3
    return torch.where((a > 0) & (i < 3 * torch.tensor(s)[a]), a, torch.zeros_like(a))


def _heads_of(state):
    """q [rows, heads, d], k and v [rows, kv_heads, d]: views into the projection's output."""
    c = state["case"]
    hq, hk = c["heads"], c["kv_heads"]
    x = state["qkv"].view(-1, hq + 2 * hk, c["dim"])
    return x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]


def _plain_rotate(state):
    c = state["case"]
    half = c["dim"] // 2
    freq = THETA ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    angle = state["positions"].double()[_axis_of_pair(c).cuda()].T * freq
    cos, sin = (f(angle).float()[:, None] for f in (torch.cos, torch.sin))
    done = []
    for x, g in zip(_heads_of(state)[:2], (state["q_norm"], state["k_norm"])):
        x = x.float()
        if g is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * g.float()
        if c["pairing"] == "half_vector":
            a, b = x[..., :half], x[..., half:]
            y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
        else:
            a, b = x[..., 0::2], x[..., 1::2]
            y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
        done.append(y.to(torch.bfloat16))
    return tuple(done)


def _copy_pages(state, source, to):
    for x in ("k", "v", "k_exp", "v_exp"):
        if state[x] is not None:
            state[x][to] = state[x][source]


def _plain_fork(state):
    table, kv, refs, page = state["table"], state["kv_len"], state["refs"], state["case"]["page"]
    src, dst = state["src"].long(), state["dst"].long()
    cols = torch.arange(table.shape[1], device="cuda")
    # The beams' sequences end: their pages' counts fall.
    old = table[dst]
    held = (cols < -(-kv[dst, None] // page)) & (old >= 0)
    refs.sub_(torch.zeros_like(refs).scatter_add_(0, torch.where(held, old, 0).long().flatten(),
                                                  held.int().flatten()))
    table[dst] = torch.where(held, -1, old)
    # Full pages are shared; a page that has room left is copied, in order, to the lowest free ones.
    length = kv[src]
    full, part = length // page, length % page != 0
    free = torch.argsort((refs > 0).to(torch.uint8), stable=True).int()
    fresh = free[(torch.cumsum(part, 0) - 1).clamp_min(0)]
    parent = table[src]
    last = parent.gather(1, full[:, None].long().clamp_max(table.shape[1] - 1))[:, 0]
    shared = (cols < full[:, None]) & (parent >= 0)
    child = torch.where(cols < full[:, None], parent, table[dst])
    child = torch.where((cols == full[:, None]) & part[:, None], fresh[:, None], child)
    table[dst] = child
    refs.scatter_add_(0, torch.where(shared, parent, 0).long().flatten(), shared.int().flatten())
    refs.scatter_add_(0, torch.where(part, fresh, 0).long(), part.int())
    kv[dst] = length
    some = part.nonzero()[:, 0]
    _copy_pages(state, last[some].long(), fresh[some].long())


def _plain_compact(state):
    table, refs, page = state["table"], state["refs"], state["case"]["page"]
    n = state["n_pages"]
    live = refs > 0
    at = torch.arange(n, device="cuda")
    end = live.sum()
    holes = (~live & (at < end)).nonzero()[:, 0]
    movers = (live & (at >= end)).nonzero()[:, 0]
    now = at.clone()
    now[movers] = holes
    refs[holes] = refs[movers]
    refs[movers] = 0
    used = torch.arange(table.shape[1], device="cuda") < -(-state["kv_len"][:, None] // page)
    table.copy_(torch.where(used & (table >= 0), now[table.long().clamp_min(0)].int(), table))
    _copy_pages(state, movers, holes)


def _values(held, exponent, pages):
    """What pages stand for, in 32 bits."""
    if exponent is None:
        return held[pages].float()
    return torch.ldexp(held[pages].view(torch.float8_e4m3fn).float(), exponent[pages].int().unsqueeze(-1) - 127)


def _bounds_of(keys):
    """Keys [..., page, d] -> (bounds [..., 2, d] as whole numbers of 2^e, exponent bytes e + 127): the largest
    and the smallest value of each channel, rounded away from the keys between them; 127 2^e covers both."""
    hi, lo = keys.amax(-2), keys.amin(-2)
    frac, ex = torch.frexp(torch.maximum(hi, -lo).amax(-1))
    e = torch.where(frac <= 127 / 128, ex - 7, ex - 6).clamp_min(-100)
    both = torch.stack((torch.ldexp(hi, -e[..., None]).ceil(), torch.ldexp(lo, -e[..., None]).floor()), -2)
    return both.to(torch.int8), (e + 127).to(torch.uint8)


def _rows_of(state):
    """Sequence and position of every row."""
    off, kv = state["row_off"].long(), state["kv_len"].long()
    r = torch.arange(state["rows"], device="cuda")
    s = torch.searchsorted(off, r, right=True) - 1
    return s, kv[s] - (off[s + 1] - r)


def _plain_bounds(state):
    s, pos = _rows_of(state)
    page = state["case"]["page"]
    done = (pos % page == page - 1).nonzero()[:, 0]      # rows that fill a page's last place
    pages = state["table"].long()[s[done], pos[done] // page]
    state["bounds"][pages], state["bounds_exp"][pages] = _bounds_of(_values(state["k"], state["k_exp"], pages))


def _shared_query(q, hk):
    """Queries [rows, heads, d] -> the group's sums of positive and of negative parts [rows, hk, 2, d], whole
    numbers: every query is rounded to a multiple of 2^e, where 1016 2^e covers what the group's sums can reach."""
    rows, hq, d = q.shape
    g = hq // hk
    q = q.float().reshape(rows, hk, g, d)
    step = 1
    while step < g:
        step *= 2
    frac, ex = torch.frexp(q.abs().amax((2, 3)) * step)
    e = torch.where(frac <= 1016 / 1024, ex - 10, ex - 9).clamp_min(-100)
    n = torch.ldexp(q, -e[..., None, None]).round()
    return torch.stack((n.clamp_min(0).sum(2), n.clamp_max(0).sum(2)), 2)


def _plain_select(state):
    c = state["case"]
    hk, page, top = c["kv_heads"], c["page"], c["top"]
    s, pos = _rows_of(state)
    w = _shared_query(_heads_of(state)[0], hk)
    own_block = pos // page
    table = state["table"].long().clamp_min(0)
    blocks = table.shape[1]
    b = state["bounds"].float()[table].permute(0, 2, 3, 4, 1)          # [n, hk, 2, d, blocks]
    e = state["bounds_exp"].int()[table].permute(0, 2, 1) - 127       # [n, hk, blocks]
    if c["n"] == 1:
        whole = (w.transpose(0, 1).flatten(2) @ b[0].flatten(1, 2)).transpose(0, 1)
    else:
        off = state["row_off"].long()
        i = torch.arange(state["max_rows"], device="cuda")
        packed = w[(off[:-1, None] + i).clamp_max(state["rows"] - 1)].transpose(1, 2).flatten(3)
        r = torch.arange(state["rows"], device="cuda")
        whole = (packed @ b.flatten(2, 3))[s, :, r - off[s]]
    score = torch.ldexp(whole, e[s] - 20)                              # exact: whole numbers under 2^24
    at = torch.arange(blocks, device="cuda")
    forced = (at < c["first"]) | (at > own_block[:, None] - c["last"])
    score = torch.where(forced[:, None], math.inf, score)
    score = torch.where((at > own_block[:, None])[:, None], -math.inf, score)
    best = torch.sort(score, dim=-1, descending=True, stable=True)[1][..., :top]
    best = torch.where(best > own_block[:, None, None], blocks, best).sort(-1)[0]
    best = torch.where(best == blocks, -1, best).int()
    return torch.nn.functional.pad(best, (0, top - best.shape[-1]), value=-1)


def _plain_attend(state):
    c = state["case"]
    d, hk, hq, page = c["dim"], c["kv_heads"], c["heads"], c["page"]
    rows, top = state["rows"], c["top"]
    s, pos = _rows_of(state)
    blocks = state["blocks"].long()
    pages = state["table"].long()[s[:, None, None], blocks.clamp_min(0)].clamp_min(0)
    head = torch.arange(hk, device="cuda")[:, None]
    whole = slice(None)
    k, v = (_values(state[x], state[x + "_exp"], whole)[pages, head].reshape(rows, hk, top * page, d)
            for x in ("k", "v"))
    key = blocks[..., None] * page + torch.arange(page, device="cuda")
    seen = ((blocks >= 0)[..., None] & (key <= pos[:, None, None, None])).reshape(rows, hk, 1, top * page)
    q = _heads_of(state)[0].float().reshape(rows, hk, hq // hk, d)
    z = (q @ k.transpose(2, 3)) * (1.0 / math.sqrt(d))
    z = z.masked_fill_(~seen, -math.inf)
    z = (z - z.amax(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)).exp_()
    o = (z @ v) / z.sum(-1, keepdim=True).clamp_min(1e-30)
    return o.reshape(rows, hq, d).to(torch.bfloat16)


# ------------------------------------------------------------------ one pass

def _handles(state):
    """What a serving loop keeps: descriptions of the cache, the pool and the call's sequences."""
    import vit_vision_encoder_gb300 as dv
    c = state["case"]
    if "kept" not in state:
        kept = {}
        if c["op"] == "rotate":
            kept["rotary"] = dv.Rotary(c["dim"], THETA, sections=_sections(c), interleaved=c["style"] == "interleaved",
                                       pairing=c["pairing"])
        else:
            kept["cache"] = dv.KvCache(state["k"], state["v"], state["k_exp"], state["v_exp"])
        if c["op"] in ("fork", "compact"):
            kept["pool"] = dv.PagePool(state["refs"], c["page"])
            kept["tables"] = dv.PageTables(state["table"], state["kv_len"])
            kept["copies"] = dv.PageCopies(state["n_pages"])
        elif c["op"] != "rotate":
            kept["chunks"] = dv.Chunks(state["row_off"], state["kv_len"], state["table"], state["max_rows"])
            kept["bounds"] = dv.KeyBounds(state["bounds"], state["bounds_exp"])
        state["kept"] = kept
    return dv, state["kept"]


def _own(state):
    c, status = state["case"], state["status"]
    dv, kept = _handles(state)
    if c["op"] == "rotate":
        q, k, _ = _heads_of(state)
        return dv.qk_norm_rope(kept["rotary"], q, k, state["positions"], state["q_norm"], state["k_norm"], EPS,
                               out=(state["q_out"], state["k_out"]))
    if c["op"] == "fork":
        dv.pages_resize(kept["pool"], kept["tables"], state["dst"], state["none"], kept["copies"], status=status)
        dv.pages_fork(kept["pool"], kept["tables"], state["src"], state["dst"], kept["copies"], status=status)
        dv.cache_copy(kept["cache"], kept["copies"], status=status)
    elif c["op"] == "compact":
        dv.pages_compact(kept["pool"], kept["tables"], kept["copies"], status=status)
        dv.cache_copy(kept["cache"], kept["copies"], status=status)
    elif c["op"] == "bounds":
        dv.cache_bounds(kept["cache"], kept["chunks"], kept["bounds"], state["rows"], status=status)
    elif c["op"] == "select":
        return dv.cache_select(kept["cache"], kept["chunks"], kept["bounds"], _heads_of(state)[0], c["top"],
                               first=c["first"], last=c["last"], out=state["blocks"], status=status)[0]
    else:
        return dv.cache_attention_blocks(kept["cache"], kept["chunks"], _heads_of(state)[0], state["blocks"],
                                         out=state["out"], status=status)[0]
    return None


def run(state):
    op = state["case"]["op"]
    if op == "compact":
        # The tables as the sequences left them, so that there is something to move in every pass.
        for x, y in zip(("table", "refs"), state["was"]):
            state[x].copy_(y)
    if own:
        got = _own(state)
    else:
        got = {"rotate": _plain_rotate, "fork": _plain_fork, "compact": _plain_compact, "bounds": _plain_bounds,
               "select": _plain_select, "attend": _plain_attend}[op](state)
    if op in ("fork", "compact"):
        # bf16 values, or e4m3 values with their exponents.
        kind = torch.bfloat16 if state["k_exp"] is None else torch.float8_e4m3fn
        got = {"table": state["table"], "kv_len": state["kv_len"], "refs": state["refs"], "k": state["k"].view(kind),
               "v": state["v"].view(kind)}
        if state["k_exp"] is not None:
            got.update(k_exp=state["k_exp"], v_exp=state["v_exp"])
    elif op == "bounds":
        got = torch.ldexp(state["bounds"].float(), state["bounds_exp"].int()[..., None, None] - 127)
    return got


# ------------------------------------------------------------------ 64 bits

def _exact_rotate(state):
    c = state["case"]
    d, half = c["dim"], c["dim"] // 2
    sections, pos = _sections(c), state["positions"].double()
    outs = []
    for x, g in zip(_heads_of(state)[:2], (state["q_norm"], state["k_norm"])):
        x = x.double()
        if g is not None:
            x = x / ((x ** 2).sum(-1, keepdim=True) / d + EPS).sqrt() * g.double()
        y = torch.empty_like(x)
        for i in range(half):
            axis = 0
            if c["style"] == "interleaved" and i % 3 and i < 3 * sections[i % 3]:
                axis = i % 3
            elif c["style"] == "sections":
                axis = 0 if i < sections[0] else 1 if i < sections[0] + sections[1] else 2
            a, b = (i, i + half) if c["pairing"] == "half_vector" else (2 * i, 2 * i + 1)
            t = (pos[axis] * math.exp(-math.log(THETA) * i / half))[:, None]
            y[..., a] = x[..., a] * t.cos() - x[..., b] * t.sin()
            y[..., b] = x[..., a] * t.sin() + x[..., b] * t.cos()
        outs.append(y)
    return tuple(outs)


def _exact_pages(state):
    """The pages after the copies (whole numbers have no value in 64 bits)."""
    c, page = state["case"], state["case"]["page"]
    kv, table, refs = (state[x].tolist() for x in ("kv_len", "table", "refs"))
    moves = []
    if c["op"] == "fork":
        free = [p for p, n in enumerate(refs) if n == 0]
        for s in state["src"].tolist():
            if kv[s] % page:
                moves.append((table[s][kv[s] // page], free[len(moves)]))
    else:
        live = sum(n > 0 for n in refs)
        moves = list(zip([p for p in range(live, len(refs)) if refs[p] > 0],
                         [p for p in range(live) if refs[p] == 0]))
    out = {x: None for x in ("table", "kv_len", "refs", "k", "v")}
    if c["kind"] == "e4m3":
        out.update(k_exp=None, v_exp=None)
    for x in ("k", "v"):
        y = state[x].double() if c["kind"] == "bf16" else state[x].view(torch.float8_e4m3fn).double()
        if moves:
            a, b = (torch.tensor(m, device="cuda") for m in zip(*moves))
            y[b] = y[a]
        out[x] = y
    return out


def _held64(state, x, pages):
    y = state[x][pages]
    if state[x + "_exp"] is None:
        return y.double()
    return y.view(torch.float8_e4m3fn).double() * torch.exp2(state[x + "_exp"][pages].double() - 127)[..., None]


def _exact_bounds(state):
    c, page = state["case"], state["case"]["page"]
    out = torch.zeros(state["bounds"].shape, dtype=torch.float64, device="cuda")
    for s, (new, kv) in enumerate(zip(*_chunks(c))):
        for b in range((kv - new) // page, kv // page):
            p = int(state["table"][s, b])
            k = _held64(state, "k", p)
            hi, lo = k.max(1)[0], k.min(1)[0]
            # 127 2^e is the least such bound at or above the block's largest magnitude
            step = torch.exp2(torch.ceil(torch.log2(k.abs().amax((1, 2)) / 127)).clamp_min(-100))[:, None]
            out[p, :, 0], out[p, :, 1] = torch.ceil(hi / step) * step, torch.floor(lo / step) * step
    return out


def _exact_attend(state):
    c = state["case"]
    d, hk, hq, page = c["dim"], c["kv_heads"], c["heads"], c["page"]
    q = _heads_of(state)[0]
    out = torch.zeros((state["rows"], hq, d), dtype=torch.float64, device="cuda")
    off, kv = state["row_off"].tolist(), state["kv_len"].tolist()
    for s in range(c["n"]):
        pages = state["table"][s, :-(-kv[s] // page)].long()
        for h in range(hk):
            k, v = (_held64(state, x, pages)[:, h].reshape(-1, d) for x in ("k", "v"))
            for r0 in range(off[s], off[s + 1], 256):
                r1 = min(off[s + 1], r0 + 256)
                p = torch.arange(r0, r1, device="cuda") + kv[s] - off[s + 1]
                picked = torch.zeros((r1 - r0, len(pages) + 1), dtype=torch.bool, device="cuda")
                b = state["blocks"][r0:r1, h].long()
                picked.scatter_(1, torch.where(b < 0, len(pages), b), True)
                seen = picked[:, :-1].repeat_interleave(page, 1)
                seen &= torch.arange(len(pages) * page, device="cuda") <= p[:, None]
                for j in range(h * (hq // hk), (h + 1) * (hq // hk)):
                    z = (q[r0:r1, j].double() @ k.T) * d ** -0.5
                    out[r0:r1, j] = torch.softmax(z.masked_fill_(~seen, -math.inf), 1) @ v
    return out


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "rotate":
        return _exact_rotate(state)
    if case["op"] in ("fork", "compact"):
        return _exact_pages(state)
    if case["op"] == "bounds":
        return _exact_bounds(state)
    if case["op"] == "select":
        return None                                       # whole numbers
    q, kv = _chunks(case)
    cost = sum(a * b for a, b in zip(q, kv)) * case["heads"] * case["dim"] * 4
    return None if cost > 8e12 else _exact_attend(state)

"""Cases of the prompt-side operators: writing a paged K/V cache, reading it
back, and the attention of a chunk of new tokens over it.

Each operator has a plain form (elementary torch operations in 32 bits) and
the framework's own call; ``own`` says which one ``run`` makes.  ``exact`` gives
the operators' definitions in 64 bits.
"""
from __future__ import annotations

import math
import random

import torch

own = False

BF16, E4M3 = 0, 1


# ------------------------------------------------------------------ cases

def _case(op, kind, dim, heads, kv_heads, page, n, chunk, history, window=0, sinks=0, mix=1, name=None):
    c = {"op": op, "kind": kind, "dim": dim, "heads": heads, "kv_heads": kv_heads, "page": page, "n": n,
         "chunk_lo": chunk[0], "chunk_hi": chunk[1], "hist_lo": history[0], "hist_hi": history[1],
         "window": window, "sinks": sinks, "mix": mix}
    if name is not None:
        c["name"] = name
    return c


def listed():
    return [
        # One new token of each of 48 running sequences: the smallest write, all latency.
        _case("write", "bf16", 128, 40, 8, 16, 48, (1, 1), (100, 4000), name="write_step_bf16"),
        # A prefill chunk of three prompts (8500 rows), quantised as it is stored.
        _case("write", "e4m3", 128, 40, 8, 64, 3, (1500, 4500), (0, 9000), mix=3, name="write_chunk_e4m3"),
        # Short prompts read back out of small pages (a hand-over to another process).
        _case("read", "bf16", 64, 16, 4, 32, 5, (1, 700), (0, 0), mix=2, name="read_short_bf16"),
        # Long prompts read back out of a quantised cache.
        _case("read", "e4m3", 128, 40, 8, 128, 4, (9000, 30000), (0, 0), mix=5, name="read_long_e4m3"),
        # One token of one sequence after an image prompt: the call whose latency a user waits for.
        _case("attention", "bf16", 128, 40, 8, 16, 1, (1, 1), (1500, 1500), name="token_one_bf16"),
        # One token of each of 32 sequences of mixed lengths.
        _case("attention", "bf16", 128, 40, 8, 64, 32, (1, 1), (400, 16000), mix=4, name="token_batch_bf16"),
        # The same with a quantised cache, more and longer sequences.
        _case("attention", "e4m3", 128, 40, 8, 64, 64, (1, 1), (2000, 30000), mix=6, name="token_batch_e4m3"),
        # Few tokens each (draft tokens being checked) behind a window of 4096 with 4 sinks.
        _case("attention", "e4m3", 128, 64, 8, 32, 24, (1, 4), (500, 60000), 4096, 4, mix=7, name="draft_window_e4m3"),
        # The span of one 1344 x 1344 image and a little text, nothing cached before.
        _case("attention", "bf16", 128, 40, 8, 64, 1, (1090, 1090), (0, 0), name="prompt_image_bf16"),
        # A chunk of a long prompt over 32k cached tokens: the largest.
        _case("attention", "bf16", 128, 40, 8, 128, 1, (2048, 2048), (32000, 32000), name="chunk_long_bf16"),
        # Short ragged chunks of several prompts, head dim 64, a window with sinks, quantised pages.
        _case("attention", "e4m3", 64, 32, 4, 32, 7, (30, 1500), (100, 20000), 1024, 5, mix=9, name="chunk_window_e4m3"),
        # A few dozen rows (the end of a prompt) over a long quantised cache.
        _case("attention", "e4m3", 128, 32, 4, 64, 2, (40, 120), (20000, 60000), mix=8, name="chunk_tail_e4m3"),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the same ranges, no dearer than the largest listed."""
    most = max(w["bytes"] + w["flops"] / 280 for w in map(work, listed()))
    while True:
        op = rng.choice(["write", "read", "attention", "attention", "attention"])
        kind = rng.choice(["bf16", "e4m3"])
        dim = rng.choice([64, 128])
        kv_heads = rng.choice([1, 2, 4, 8, 8, 10])
        heads = kv_heads * rng.choice([1, 2, 4, 5, 7, 8, 16])
        page = rng.choice([16, 32, 64, 128])
        n = _log_uniform(rng, 1, 64)
        form = rng.choice(["token", "token", "draft", "chunk", "chunk", "prompt"])
        window, sinks = rng.choice([(0, 0), (0, 0), (_log_uniform(rng, 100, 5000), rng.choice([0, 1, 4, 16, 37]))])
        hist_hi = _log_uniform(rng, 20, 60000)
        hist_lo = _log_uniform(rng, 1, hist_hi)
        if op == "read":
            lo = _log_uniform(rng, 1, 20000)
            chunk, history, window, sinks = (lo, _log_uniform(rng, lo, 30000)), (0, 0), 0, 0
        else:
            if op == "write":
                window, sinks = 0, 0
            if form == "token":
                chunk = (1, 1)
            elif form == "draft":
                chunk = (1, _log_uniform(rng, 2, 9))
            else:
                lo = _log_uniform(rng, 8, 3000)
                chunk = (lo, _log_uniform(rng, lo, 4000))
            history = (0, 0) if form == "prompt" else (hist_lo, hist_hi)
        c = _case(op, kind, dim, heads, kv_heads, page, n, chunk, history, window, sinks, rng.randrange(1, 1 << 30))
        w = work(c)
        # The plain form pads every sequence to the longest: keep that, and the inputs, within a few GB.
        q, kv = _lengths(c)
        padded = n * max(kv) * kv_heads * dim * 8
        scores = n * heads * max(q) * max(kv) * 4 if op == "attention" else 0
        made = sum(q) * (heads + 2 * kv_heads) * dim * 4
        if w["bytes"] + w["flops"] / 280 <= most and padded < 20e9 and scores < 12e9 and made < 4e9:
            return c


def _lengths(case):
    """New tokens and cached tokens (those included) of each sequence."""
    r = random.Random(case["mix"])

    def between(lo, hi):
        return lo if lo == hi else _log_uniform(r, max(lo, 1), hi)

    q = [between(case["chunk_lo"], case["chunk_hi"]) for _ in range(case["n"])]
    kv = [c + between(case["hist_lo"], case["hist_hi"]) for c in q]
    return q, kv


def _visible(case, c, kv):
    """(sum over the rows of the keys each sees, keys that any row sees) of one sequence."""
    w, s = case["window"], case["sinks"]
    total = 0
    for i in (range(c) if w else ()):
        p = kv - c + i
        lo = max(0, p - w + 1)
        total += p + 1 - lo + min(s, lo)
    if not w:
        total = c * (kv - c) + c * (c + 1) // 2
        return total, kv
    lo = max(0, kv - c - w + 1)
    return total, kv - lo + min(s, lo)


def work(case):
    q, kv = _lengths(case)
    rows, d, hk = sum(q), case["dim"], case["kv_heads"]
    held = 2 * d if case["kind"] == "bf16" else d + 1      # bytes of one key or value
    if case["op"] in ("write", "read"):
        return {"bytes": rows * hk * 2 * (2 * d + held) + 4 * rows / case["page"], "flops": rows * hk * 2 * d}
    pairs = seen = 0
    for c, l in zip(q, kv):
        a, b = _visible(case, c, l)
        pairs += a
        seen += b
    return {"bytes": rows * case["heads"] * d * 4 + seen * hk * 2 * held + 4 * seen / case["page"],
            "flops": 4.0 * pairs * d * case["heads"]}


# ------------------------------------------------------------------ inputs

def _rows(shape, gen, channel):
    """Keys or values as a projection leaves them: unequal channels, a few large ones."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    return (x * channel).to(torch.bfloat16)


def _quantise(x):
    """bf16 rows [..., d] -> (float8 values of x 2^-e, exponent bytes e + 127)."""
    top = x.float().abs().amax(-1)
    frac, ex = torch.frexp(top)
    e = torch.where(frac <= 0.875, ex - 9, ex - 8).clamp_min(-117)
    fine = torch.isfinite(top)
    scaled = torch.ldexp(x.float(), -e.unsqueeze(-1))
    scaled = torch.where(fine.unsqueeze(-1), scaled, torch.full_like(scaled, math.nan))
    return scaled.to(torch.float8_e4m3fn), torch.where(fine, e + 127, torch.full_like(e, 255)).to(torch.uint8)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    q, kv = _lengths(case)
    n, d, hk, hq, page = case["n"], case["dim"], case["kv_heads"], case["heads"], case["page"]
    rows = sum(q)
    cols = -(-max(kv) // page)
    used = [-(-l // page) for l in kv]
    n_pages = sum(used) + 3
    order = torch.randperm(n_pages, generator=gen, device="cuda").to(torch.int32)
    # Columns past a sequence's last page hold -1, as a block allocator leaves them.
    table = torch.full((n, cols), -1, dtype=torch.int32, device="cuda")
    at = 0
    for s, u in enumerate(used):
        table[s, :u] = order[at:at + u]
        at += u
    channel = torch.exp(0.4 * torch.randn((hk, 1, d), generator=gen, device="cuda"))
    state = {"case": case, "rows": rows, "table": table, "max_rows": max(q), "n_pages": n_pages,
             "row_off": torch.tensor([sum(q[:i]) for i in range(n + 1)], dtype=torch.int32, device="cuda"),
             "kv_len": torch.tensor(kv, dtype=torch.int32, device="cuda"),
             "status": torch.zeros(1, dtype=torch.int32, device="cuda"),
             "k_exp": None, "v_exp": None}
    # q, k and v of the new tokens side by side, as one projection writes them.
    qkv = torch.randn((rows, (hq + 2 * hk) * d), generator=gen, device="cuda").to(torch.bfloat16)
    state["qkv"] = qkv
    pages = (n_pages, hk, page, d)
    if case["op"] == "write":
        qkv[:, hq * d:] = (qkv[:, hq * d:].float().view(rows, 2, hk, d) * channel.view(1, 1, hk, d)).view(
            rows, -1).to(torch.bfloat16)
        kind = torch.bfloat16 if case["kind"] == "bf16" else torch.uint8
        state["k"], state["v"] = (torch.zeros(pages, dtype=kind, device="cuda") for _ in range(2))
        if case["kind"] == "e4m3":
            state["k_exp"], state["v_exp"] = (torch.zeros(pages[:3], dtype=torch.uint8, device="cuda")
                                              for _ in range(2))
    else:
        for x in ("k", "v"):
            held = _rows(pages, gen, channel)
            if case["kind"] == "e4m3":
                bits, state[x + "_exp"] = _quantise(held)
                held = bits.view(torch.uint8)
            state[x] = held
    if case["op"] == "attention":
        state["out"] = torch.zeros((rows, hq, d), dtype=torch.bfloat16, device="cuda")
    if case["op"] == "read":
        state["out_k"], state["out_v"] = (torch.zeros((rows, hk, d), dtype=torch.bfloat16, device="cuda")
                                          for _ in range(2))
    return state


def _split(state):
    """q [rows, heads, d], k and v [rows, kv_heads, d]: views into the projection's output."""
    c = state["case"]
    hq, hk, d = c["heads"], c["kv_heads"], c["dim"]
    x = state["qkv"].view(state["rows"], hq + 2 * hk, d)
    return x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]


# ------------------------------------------------------------------ the operators

def _places(state):
    """Sequence, position, page and slot of every row."""
    off, kv, page = state["row_off"].long(), state["kv_len"].long(), state["case"]["page"]
    r = torch.arange(state["rows"], device="cuda")
    s = torch.searchsorted(off, r, right=True) - 1
    pos = kv[s] - (off[s + 1] - r)
    return s, pos, state["table"].long()[s, pos // page], pos % page


def _values(held, exponent):
    """What the cache's contents stand for, in 32 bits."""
    if exponent is None:
        return held.float()
    return torch.ldexp(held.view(torch.float8_e4m3fn).float(), exponent.int().unsqueeze(-1) - 127)


def _plain_write(state):
    _, k, v = _split(state)
    _, _, page, slot = _places(state)
    if state["k_exp"] is None:
        state["k"][page, :, slot] = k
        state["v"][page, :, slot] = v
        return
    for x, name in ((k, "k"), (v, "v")):
        bits, ex = _quantise(x)
        state[name][page, :, slot] = bits.view(torch.uint8)
        state[name + "_exp"][page, :, slot] = ex


def _plain_read(state):
    _, _, page, slot = _places(state)
    return tuple(_values(state[x][page, :, slot], None if state[x + "_exp"] is None else
                         state[x + "_exp"][page, :, slot]).to(torch.bfloat16) for x in ("k", "v"))


def _plain_attention(state):
    c = state["case"]
    n, d, hk, hq, page = c["n"], c["dim"], c["kv_heads"], c["heads"], c["page"]
    g, mq = hq // hk, state["max_rows"]
    table = state["table"].long().clamp_min(0)
    length = table.shape[1] * page
    off, kv = state["row_off"].long(), state["kv_len"].long()

    def cached(x):
        e = state[x + "_exp"]
        y = _values(state[x][table], None if e is None else e[table])
        return y.permute(0, 2, 1, 3, 4).reshape(n, hk, length, d)

    i = torch.arange(mq, device="cuda")
    j = torch.arange(length, device="cuda")
    q = _split(state)[0][(off[:-1, None] + i).clamp_max(state["rows"] - 1)].float()
    q = q.view(n, mq, hk, g, d).permute(0, 2, 3, 1, 4).reshape(n, hk, g * mq, d)
    s = (q @ cached("k").transpose(2, 3)).mul_(1.0 / math.sqrt(d)).view(n, hk, g, mq, length)
    pos = (kv - (off[1:] - off[:-1]))[:, None] + i
    seen = j <= pos[..., None]
    if c["window"]:
        seen = seen & ((j > pos[..., None] - c["window"]) | (j < c["sinks"]))
    seen = (seen & (j < kv[:, None, None]))[:, None, None]
    s.masked_fill_(~seen, -math.inf)
    s.sub_(s.amax(-1, keepdim=True).clamp_min(torch.finfo(torch.float32).min)).exp_()
    total = s.sum(-1, keepdim=True)
    v = torch.where((j < kv[:, None])[:, None, :, None], cached("v"), torch.zeros((), device="cuda"))
    o = (s.view(n, hk, g * mq, length) @ v).view(n, hk, g, mq, d)
    o = torch.where(total > 0, o / total, torch.zeros((), device="cuda"))
    r = torch.arange(state["rows"], device="cuda")
    at = torch.searchsorted(off, r, right=True) - 1
    return o[at, :, :, r - off[at]].reshape(state["rows"], hq, d).to(torch.bfloat16)


def _own_handles(state):
    """The cache and the chunk description that a serving loop keeps."""
    import vit_vision_encoder_gb300 as dv
    if "cache" not in state:
        state["cache"] = dv.KvCache(state["k"], state["v"], state["k_exp"], state["v_exp"])
        state["chunks"] = dv.Chunks(state["row_off"], state["kv_len"], state["table"], state["max_rows"])
    return dv, state["cache"], state["chunks"]


def run(state):
    op = state["case"]["op"]
    if own:
        dv, cache, chunks = _own_handles(state)
        q, k, v = _split(state)
        if op == "write":
            dv.cache_write(cache, chunks, k, v, status=state["status"])
        elif op == "read":
            return dv.cache_read(cache, chunks, state["rows"], out=(state["out_k"], state["out_v"]),
                                 status=state["status"])[:2]
        else:
            return dv.cache_attention(cache, chunks, q, window=state["case"]["window"], sinks=state["case"]["sinks"],
                                      out=state["out"], status=state["status"])[0]
    elif op == "write":
        _plain_write(state)
    elif op == "read":
        return _plain_read(state)
    else:
        return _plain_attention(state)
    # The cache itself: bf16 values, or e4m3 values with their exponents.
    if state["k_exp"] is None:
        return state["k"], state["v"]
    return (state["k"].view(torch.float8_e4m3fn), state["v"].view(torch.float8_e4m3fn), state["k_exp"],
            state["v_exp"])


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    state = prepare(case, seed)
    off, kv, table = (state[x].tolist() for x in ("row_off", "kv_len", "table"))
    page, d, hk = case["page"], case["dim"], case["kv_heads"]
    q, k, v = _split(state)

    def slots(s, count):
        """Flat (page, slot) numbers of the positions 0 .. count - 1 of sequence s."""
        j = torch.arange(count)
        return torch.tensor(table[s])[j // page].cuda(), (j % page).cuda()

    def held(x, s, count):
        p, o = slots(s, count)
        y = state[x][p, :, o]
        if state[x + "_exp"] is None:
            return y.double()
        y = y.view(torch.float8_e4m3fn).double()
        return y * torch.exp2(state[x + "_exp"][p, :, o].double() - 127)[..., None]

    if case["op"] == "write":
        outs = []
        for x, name in ((k, "k"), (v, "v")):
            to = torch.zeros((state["n_pages"], hk, page, d), dtype=torch.float64, device="cuda")
            for s in range(case["n"]):
                p, o = slots(s, kv[s])
                new = off[s + 1] - off[s]
                y = x[off[s]:off[s + 1]].double()
                if case["kind"] == "e4m3":
                    # 448 2^e is the least such bound at or above the row's largest magnitude
                    top = y.abs().amax(-1, keepdim=True)
                    y = y / torch.exp2(torch.ceil(torch.log2(top / 448)).clamp_min(-117))
                to[p[kv[s] - new:], :, o[kv[s] - new:]] = y
            outs.append(to)
        return tuple(outs) if case["kind"] == "bf16" else (*outs, None, None)
    if case["op"] == "read":
        return tuple(torch.cat([held(x, s, kv[s])[kv[s] - (off[s + 1] - off[s]):] for s in range(case["n"])])
                     for x in ("k", "v"))
    g = case["heads"] // hk
    out = torch.zeros((state["rows"], case["heads"], d), dtype=torch.float64, device="cuda")
    for s in range(case["n"]):
        new = off[s + 1] - off[s]
        ks, vs = held("k", s, kv[s]), held("v", s, kv[s])
        p = torch.arange(kv[s] - new, kv[s], device="cuda")[:, None]
        j = torch.arange(kv[s], device="cuda")[None]
        hidden = j > p
        if case["window"]:
            hidden = hidden | ((j <= p - case["window"]) & (j >= case["sinks"]))
        for h in range(case["heads"]):
            z = (q[off[s]:off[s + 1], h].double() @ ks[:, h // g].T) * d ** -0.5
            z[hidden] = -math.inf
            out[off[s]:off[s + 1], h] = torch.softmax(z, 1) @ vs[:, h // g]
    return out

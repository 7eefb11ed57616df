"""Bounds of a cache's pages, the selection of blocks by them and attention over listed
blocks on the GPU, against plain implementations in whole numbers and in 64 bits, and
a long prompt taken through all of them."""
import math

import numpy as np
import pytest

from test_gpu_cache import Setup, check_attention, f64, quantise

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def dv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import vit_vision_encoder_gb300
    return vit_vision_encoder_gb300


# ------------------------------------------------------------------ the definitions

def least(a, times, floor=-100):
    """The least e >= floor with a <= times 2^e (exact: a and 2^e are floats)."""
    e = floor
    while a > times * 2.0 ** e:
        e += 1
    return e


def bounds64(keys):
    """Keys [page, dim] -> (H, L, exponent byte)."""
    if not np.isfinite(keys).all():
        return None, None, 255
    e = least(np.abs(keys).max(), 127)
    return np.ceil(keys.max(0) / 2.0 ** e), np.floor(keys.min(0) / 2.0 ** e), e + 127


def all_bounds(st, n_pages=None):
    """Bounds of every page of a Setup, whatever is in it."""
    k = st.held()[0]
    hi_lo = np.zeros((st.n_pages, st.kv_heads, 2, st.dim), dtype=np.int8)
    exp = np.zeros((st.n_pages, st.kv_heads), dtype=np.uint8)
    for p in range(st.n_pages):
        for h in range(st.kv_heads):
            hi, lo, e = bounds64(k[p, h])
            exp[p, h] = e
            if e != 255:
                hi_lo[p, h] = hi, lo
    return hi_lo, exp


def lists64(st, hi_lo, exp, q, top, first, last):
    """The lists of every row, None for rows of no sequence: whole numbers throughout."""
    q = f64(q)
    g = q.shape[1] // st.kv_heads
    G = 1
    while G < g:
        G *= 2
    out = [None] * st.rows
    table = st.chunks.table.cpu().numpy()
    for s in range(len(st.q)):
        for i in range(st.q[s]):
            r, p = st.off[s] + i, st.kv[s] - st.q[s] + i
            out[r] = np.full((st.kv_heads, top), -1)
            own = p // st.page
            for h in range(st.kv_heads if p >= 0 else 0):
                x = q[r, h * g:(h + 1) * g]
                plus = minus = np.zeros(st.dim)
                if np.isfinite(x).all():
                    n = np.rint(x / 2.0 ** least(np.abs(x).max() * G, 1016))
                    plus, minus = np.maximum(n, 0).sum(0), np.minimum(n, 0).sum(0)
                key = []
                for b in range(own + 1):
                    page = int(table[s, b])
                    if page < 0:
                        continue
                    if b < first or b > own - last:
                        score = math.inf
                    elif exp[page, h] == 255:
                        score = 1e300
                    else:
                        whole = int((plus * hi_lo[page, h, 0] + minus * hi_lo[page, h, 1]).sum())
                        assert abs(whole) < 2 ** 24
                        score = whole * 2.0 ** (int(exp[page, h]) - 127)
                    key.append((-score, b))
                best = sorted(b for _, b in sorted(key)[:top])
                out[r][h, :len(best)] = best
    return out


def make(dv, q, kv, kv_heads, dim, page, kind, **kw):
    st = Setup(dv, q, kv, kv_heads, dim, page, kind, **kw)
    st.bounds = dv.KeyBounds.empty(st.cache)
    hi_lo, exp = all_bounds(st)
    st.hi_lo, st.exp = hi_lo, exp
    st.bounds.hi_lo.copy_(torch.from_numpy(hi_lo))
    st.bounds.exp.copy_(torch.from_numpy(exp))
    return st


# ------------------------------------------------------------------ bounds

@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("page,dim,kv_heads", [(16, 64, 1), (16, 128, 8), (32, 64, 3), (64, 128, 10), (128, 64, 2),
                                               (128, 128, 4)])
def test_bounds(dv, kind, page, dim, kv_heads):
    """Every block that a row completes, and no other; partly filled and older ones stay."""
    q = [1, 1, page, 3 * page + 5, 0, 2, 7, page - 1, 1]
    kv = [page, page + 1, page, 5 * page + 2, 2 * page, 4 * page + 1, 3, 2 * page - 1, 3 * page]
    st = Setup(dv, q, kv, kv_heads, dim, page, kind, seed=page + dim, back=3)
    b = dv.KeyBounds.empty(st.cache)
    b.hi_lo.fill_(77)
    b.exp.fill_(3)
    status = dv.cache_bounds(st.cache, st.chunks, b, st.rows)
    torch.cuda.synchronize()
    assert int(status.item()) == dv.OK
    hi_lo, exp = all_bounds(st)
    done = np.zeros(st.n_pages, dtype=bool)
    for s in range(len(q)):
        for j in range(max(kv[s] - q[s], 0) // page, kv[s] // page):
            done[int(st.table[s, j])] = True
    got, got_exp = b.hi_lo.cpu().numpy(), b.exp.cpu().numpy()
    assert np.array_equal(got[done], hi_lo[done]) and np.array_equal(got_exp[done], exp[done])
    assert (got[~done] == 77).all() and (got_exp[~done] == 3).all()


def test_bounds_of_extreme_keys(dv):
    page, dim = 16, 64
    st = Setup(dv, [160], [160], 1, dim, page, "bf16")
    k = st.cache.k
    for j, v in enumerate([0.0, 3.3e38, 1e-38, 1e-40, math.inf, -math.inf, math.nan, 127 * 2.0 ** 5, 127.5 * 2.0 ** 5]):
        k[int(st.table[0, j])] *= 0.01 if v == 0 or abs(v) > 100 else 0.0
        k[int(st.table[0, j]), 0, 5, 9] = v
    k[int(st.table[0, 0])] = 0
    k[int(st.table[0, 1]), 0, 3] = -3.3e38
    b = dv.KeyBounds.empty(st.cache)
    status = dv.cache_bounds(st.cache, st.chunks, b, st.rows)
    torch.cuda.synchronize()
    hi_lo, exp = all_bounds(st)
    used = st.table[0, :10].numpy()
    assert int(status.item()) == dv.OK
    assert np.array_equal(b.exp.cpu().numpy()[used], exp[used])
    assert np.array_equal(b.hi_lo.cpu().numpy()[used], hi_lo[used])
    assert (exp[used[4:7]] == 255).all() and exp[used[0]] == 27


@pytest.mark.parametrize("kind,large,small", [("bf16", 3.3e38, 1e-9), ("bf16", 1e30, 1e-18), ("bf16", 3.0, 2.0 ** -133),
                                              ("bf16", 2.0 ** 120, 2.0 ** -100), ("e4m3", 1e30, 1e-18),
                                              ("e4m3", 200 * 2.0 ** 120, 2.0 ** -110), ("e4m3", 3.3e38, 1e-9)])
def test_bounds_of_magnitudes_far_apart(dv, kind, large, small):
    """A channel so small beside the block's largest value that their ratio is no float has its bound a step from 0."""
    page, dim = 16, 64
    st = Setup(dv, [64], [64], 1, dim, page, kind, seed=6)
    x = np.zeros((st.n_pages, 1, page, dim))
    for j, sign in enumerate((1, -1, 1, -1)):
        p = int(st.table[0, j])
        x[p, 0, 3, 5] = large * (1 if j < 2 else -1)
        x[p, 0, :, 9:40:3] = sign * small            # the channel has no other sign
        if kind == "e4m3":
            x[p, 0, 3, 9:40:3] = 0                   # one exponent a key
        x[p, 0, 7, 41], x[p, 0, 8, 41] = small, -small
    if kind == "bf16":
        st.cache.k.copy_(torch.from_numpy(x).bfloat16())
    else:
        b, e = quantise(torch.from_numpy(x).bfloat16().double().numpy())
        st.cache.k.copy_(torch.from_numpy(b))
        st.cache.k_exp.copy_(torch.from_numpy(e))
    b = dv.KeyBounds.empty(st.cache)
    status = dv.cache_bounds(st.cache, st.chunks, b, st.rows)
    torch.cuda.synchronize()
    hi_lo, exp = all_bounds(st)
    used = st.table[0, :4].numpy()
    assert int(status.item()) == dv.OK and (exp[used] < 255).all()
    assert (hi_lo[used[::2], 0, 0, 9] == 1).all() and (hi_lo[used[1::2], 0, 1, 9] == -1).all()
    assert np.array_equal(b.exp.cpu().numpy()[used], exp[used])
    assert np.array_equal(b.hi_lo.cpu().numpy()[used], hi_lo[used])


def test_bounds_hold_every_key(dv):
    """H and L enclose the keys they stand for."""
    for kind in ("bf16", "e4m3"):
        st = make(dv, [300], [300], 2, 128, 32, kind)
        k = st.held()[0]
        step = 2.0 ** (st.exp.astype(float) - 127)[..., None]
        assert (st.hi_lo[:, :, 0] * step >= k.max(2)).all() and (st.hi_lo[:, :, 1] * step <= k.min(2)).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("group,dim", [(1, 128), (5, 64), (128, 64)])
def test_written_bounds_and_scores_from_above(dv, kind, group, dim):
    """What ds_vit_cache_bounds writes holds every key, and the score from it lies at or over the true sum of products with
    every key of the block, but for what the rounding of the queries to whole numbers moves."""
    page, heads = 16, 2
    st = Setup(dv, [330], [330], heads, dim, page, kind, seed=group)
    b = dv.KeyBounds.empty(st.cache)
    status = dv.cache_bounds(st.cache, st.chunks, b, st.rows)
    torch.cuda.synchronize()
    assert int(status.item()) == dv.OK
    used = st.table[0, :330 // page].numpy()             # the last block is not full
    k = st.held()[0][used]
    step = 2.0 ** (b.exp.cpu().numpy()[used].astype(float) - 127)[..., None]
    hi, lo = (b.hi_lo.cpu().numpy()[used, :, i] * step for i in range(2))
    assert (hi >= k.max(2)).all() and (lo <= k.min(2)).all()
    assert (hi < k.max(2) + step).all() and (lo > k.min(2) - step).all()
    q = f64(st.queries(heads * group))[::29]
    G = 1 << (group - 1).bit_length()
    for x in q.reshape(-1, heads, group, dim):
        for h in range(heads):
            unit = 2.0 ** least(np.abs(x[h]).max() * G, 1016)
            n = np.rint(x[h] / unit)
            score = unit * (hi[:, h] @ np.maximum(n, 0).sum(0) + lo[:, h] @ np.minimum(n, 0).sum(0))
            moved = np.abs(k[:, h]).max(1) @ np.abs(x[h] - unit * n).sum(0)
            true = (k[:, h] @ x[h].sum(0)).max(1)
            assert (true <= score + moved + 1e-9 * np.abs(score)).all()


# ------------------------------------------------------------------ selection

@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("group", [1, 5, 128])
@pytest.mark.parametrize("n,rows", [(12, 1), (1, 300)])
def test_the_block_of_a_matching_key_is_chosen(dv, kind, group, n, rows):
    """Each row's queries lie near one key, twenty times as long, of one block, other blocks hold such keys of other rows:
    the block is listed."""
    heads, dim, page, kv, top = 4, 64, 16, 2000, 4
    g = torch.Generator().manual_seed(group + n)
    many = 50 if n == 1 else 3                           # directions of a sequence, each with a block of its own
    base = torch.randn((n, many, heads, dim), generator=g)
    block = torch.stack([torch.randperm(100, generator=g)[:many] for _ in range(n)])
    k = torch.randn((n, kv, heads, dim), generator=g)
    for s in range(n):
        at = block[s] * page + torch.randint(0, page, (many,), generator=g)
        k[s, at] = 20 * base[s]
    cache = dv.KvCache.empty(n * kv // page, heads, page, dim, dv.CACHE_BF16 if kind == "bf16" else dv.CACHE_E4M3)
    table = torch.randperm(n * kv // page, generator=g).int().view(n, -1).cuda()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")   # noqa: E731
    whole = dv.Chunks(i32([kv * s for s in range(n + 1)]), i32([kv] * n), table, kv)
    status = dv.cache_write(cache, whole, *[k.view(n * kv, heads, dim).bfloat16().cuda()] * 2)
    bounds = dv.KeyBounds.empty(cache)
    dv.cache_bounds(cache, whole, bounds, n * kv, status)
    which = torch.randint(0, many, (n, rows), generator=g)
    q = torch.stack([base[s, which[s]] for s in range(n)]).view(n * rows, heads, 1, dim)
    q = (q + 0.2 * torch.randn((n * rows, heads, group, dim), generator=g)).view(n * rows, heads * group, dim)
    chunks = dv.Chunks(i32([rows * s for s in range(n + 1)]), i32([kv] * n), table, rows)
    got, _ = dv.cache_select(cache, chunks, bounds, q.bfloat16().cuda(), top, 0, 1, status=status)
    torch.cuda.synchronize()
    want = torch.stack([block[s, which[s]] for s in range(n)]).view(n * rows, 1, 1)
    assert int(status.item()) == dv.OK and (got.cpu() == want).any(-1).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_a_chunk_beside_single_rows(dv, kind):
    """A prompt's chunk, draft tokens and single tokens of many sequences in one call: tiles of packed rows that hold up
    to sixteen sequences, as the call has more rows than CTAs' worth."""
    q = [1] * 13 + [40] + [1] * 30 + [0, 9] + [1] * 20
    kv = [17 + 37 * i % 900 for i in range(13)] + [700] + [1 + 211 * i % 1000 for i in range(30)] + [64, 300]
    kv += [16 * i + 16 for i in range(20)]
    st = make(dv, q, kv, 8, 64, 16, kind, seed=2, front=1, back=3)
    assert st.rows * 8 > 4 * torch.cuda.get_device_properties(0).multi_processor_count
    x = st.queries(16)
    for top in (5, 40):
        got = check_select(dv, st, 16, top, 1, 2, q=x)
    blocks = torch.from_numpy(got).int()
    blocks[:, :, 6:] = -1
    check_blocks(dv, st, 16, blocks, q=x)


def check_select(dv, st, heads, top, first, last, q=None):
    q = st.queries(heads) if q is None else q
    out = torch.full((st.rows, st.kv_heads, top), -7, dtype=torch.int32, device="cuda")
    got, status = dv.cache_select(st.cache, st.chunks, st.bounds, q, top, first, last, out=out)
    torch.cuda.synchronize()
    assert int(status.item()) == dv.OK
    got = got.cpu().numpy()
    for r, want in enumerate(lists64(st, st.hi_lo, st.exp, q, top, first, last)):
        if want is None:
            assert (got[r] == -7).all()
        else:
            assert np.array_equal(got[r], want), (r, got[r], want)
    return got


SELECT = [
    # q, kv, kv_heads, dim, page, heads, top, first, last
    ([1], [1], 1, 64, 16, 1, 1, 0, 1),
    ([1], [1000], 8, 128, 16, 40, 8, 1, 2),
    ([1, 1, 1], [17, 900, 333], 2, 64, 32, 10, 5, 1, 1),
    ([1] * 40, [50 * i + 1 for i in range(40)], 1, 128, 16, 7, 6, 0, 2),
    ([3, 0, 5, 8], [200, 40, 5, 600], 3, 128, 16, 3, 9, 2, 3),        # draft tokens, a sequence without rows
    ([700], [700], 4, 64, 16, 64, 12, 1, 2),                          # a prompt, more rows than there are CTAs' worth
    ([123, 9, 251], [1000, 9, 700], 4, 128, 16, 20, 7, 1, 1),         # tiles of rows across sequences
    ([20], [300], 1, 64, 16, 128, 40, 0, 1),                          # more places than blocks; the largest group
    ([30], [25], 2, 64, 16, 4, 3, 1, 1),                              # front padding
    ([1], [9000], 2, 64, 16, 8, 300, 5, 9),
    ([1, 1], [20000, 19000], 1, 64, 16, 5, 33, 1, 1),                 # more than a thousand blocks
    ([260], [3000], 4, 64, 16, 4, 40, 1, 2),                          # many rows: more than 32 of 187, more than 128, ...
    ([260], [3000], 4, 64, 16, 4, 128, 1, 2),
    ([260], [3000], 4, 64, 16, 4, 150, 0, 1),
    ([260], [3000], 4, 64, 16, 4, 20, 9, 11),                         # ... nothing but forced ones
    ([300], [9000], 3, 64, 16, 3, 100, 1, 2),                         # 562 blocks
    ([1], [9000], 2, 64, 16, 8, 100, 60, 40),                         # one row: nothing but forced ones
    ([1], [9000], 2, 64, 16, 8, 256, 1, 1),
    ([1], [9000], 2, 64, 16, 8, 257, 1, 1),
]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("case", range(len(SELECT)))
def test_select(dv, case, kind):
    q, kv, kv_heads, dim, page, heads, top, first, last = SELECT[case]
    st = make(dv, q, kv, kv_heads, dim, page, kind, seed=case, front=2, back=5)
    check_select(dv, st, heads, top, first, last)


def test_select_ties_go_to_the_lowest_block(dv):
    for q, kv in (([1], [640]), ([600], [640])):
        st = make(dv, q, kv, 4, 64, 16, "bf16")
        st.bounds.hi_lo.fill_(5)
        st.bounds.exp.fill_(120)
        st.hi_lo[:], st.exp[:] = 5, 120
        check_select(dv, st, 8, 6, 1, 1)
        st.hi_lo[::3], st.exp[::3] = 10, 119            # the same scores in another form
        st.hi_lo[1::3] = 4
        st.bounds.hi_lo.copy_(torch.from_numpy(st.hi_lo))
        st.bounds.exp.copy_(torch.from_numpy(st.exp))
        check_select(dv, st, 8, 6, 1, 1)
        check_select(dv, st, 8, 20, 0, 1, q=torch.zeros((st.rows, 8, 64), dtype=torch.bfloat16, device="cuda"))
    for q, kv in (([1], [9000]), ([200], [5000])):      # more of a kind than the lists in between hold
        st = make(dv, q, kv, 4, 64, 16, "bf16")
        for few in (0, 3):
            st.exp[:], st.hi_lo[:] = 120, 5
            if few:
                st.hi_lo[::few] = 6
            st.bounds.hi_lo.copy_(torch.from_numpy(st.hi_lo))
            st.bounds.exp.copy_(torch.from_numpy(st.exp))
            for top in (6, 33, 70, 130, 300):
                check_select(dv, st, 8, top, 2, 2)


def test_select_over_extremes(dv):
    """Far exponents, blocks and rows that are not finite, pages given away."""
    for q, kv in (([2, 1], [400, 333]), ([390], [400])):
        st = make(dv, q, kv, 2, 64, 16, "bf16", seed=3)
        r = np.random.default_rng(1)
        st.exp[:] = r.choice([27, 60, 127, 200, 249, 255], st.exp.shape)
        st.hi_lo[:] = r.integers(-127, 128, st.hi_lo.shape)
        st.bounds.hi_lo.copy_(torch.from_numpy(st.hi_lo))
        st.bounds.exp.copy_(torch.from_numpy(st.exp))
        x = st.queries(6)
        x = x.clone()
        x[0, 1, 7] = math.inf
        x[1, 4] *= 1e30
        x[-1] *= 1e-25
        check_select(dv, st, 6, 7, 1, 2, q=x)
        st.chunks.table[0, 3:9] = -1
        check_select(dv, st, 6, 7, 5, 2, q=x)
        st.chunks.table[0, 2] = st.n_pages               # no page of the cache: reported, not taken
        out, status = dv.cache_select(st.cache, st.chunks, st.bounds, x, 7, 5, 2)
        torch.cuda.synchronize()
        assert int(status.item()) == dv.ERANGE and not (out[0] == 2).any()


def test_select_sums_at_their_limit(dv):
    """Shared queries of up to 1024 in every channel and bounds of 125 to 127: sums within a percent of 2^24 that
    differ in their last bits."""
    for q, kv in (([1], [900]), ([200], [900])):
        st = make(dv, q, kv, 4, 128, 16, "bf16", seed=5)
        r = np.random.default_rng(2)
        st.hi_lo[:, :, 0] = r.integers(125, 128, st.hi_lo[:, :, 0].shape)
        st.hi_lo[:, :, 1] = -r.integers(125, 128, st.hi_lo[:, :, 1].shape)
        st.exp[:] = 120
        st.bounds.hi_lo.copy_(torch.from_numpy(st.hi_lo))
        st.bounds.exp.copy_(torch.from_numpy(st.exp))
        x = np.full((st.rows, 256, 128), 15.875)         # 64 heads of 16 when rounded
        x[:, ::64] = r.integers(12, 16, (st.rows, 4, 128))
        x[:, 1] = 15.875                                 # the exponent's
        x[1::3] *= -1
        x[2::3] *= r.choice([-1, 1], x[2::3, :1].shape)
        check_select(dv, st, 256, 9, 1, 1, q=torch.from_numpy(x).bfloat16().cuda())
        check_select(dv, st, 256, 40, 1, 1, q=torch.from_numpy(x).bfloat16().cuda())


def test_select_in_wide_tables(dv):
    """Rows share their loads in smaller groups as the table gets wider."""
    for cols in (3000, 9000, 20000, dv.SELECT_MAX_COLS):
        st = make(dv, [200], [500], 8, 64, 16, "bf16", cols=cols)
        check_select(dv, st, 8, 5, 1, 1)
    st = make(dv, [1], [500], 8, 64, 16, "bf16", cols=dv.SELECT_MAX_COLS + 1)
    with pytest.raises(dv.DsVitError):
        dv.cache_select(st.cache, st.chunks, st.bounds, st.queries(8), 5)


@pytest.mark.parametrize("dim", [64, 128])
def test_select_longer_lists_in_wide_tables(dv, dim):
    """Tables on both sides of the widths at which two CTAs, with the keys that they hold for longer lists, fit an SM."""
    st = make(dv, [200], [700], 8, dim, 16, "bf16", cols=700)
    for cols in (1376, 1408, 1440, 1500, 1568, 1600, 1632, 1800):
        st.chunks = dv.Chunks(st.chunks.row_off, st.chunks.kv_len,
                              torch.nn.functional.pad(st.table, (0, cols - st.table.shape[1]), value=-1).cuda(), 200)
        for top in (32, 33):
            check_select(dv, st, 8, top, 1, 1)


def test_select_long_contexts(dv):
    """Many thousand blocks against the same whole numbers in torch (one sequence, one head)."""
    page, dim, blocks = 16, 64, 30011
    g = torch.Generator().manual_seed(0)
    cache = dv.KvCache.empty(blocks, 1, page, dim)
    hi_lo = torch.randint(-127, 128, (blocks, 1, 2, dim), generator=g).to(torch.int8)
    exp = torch.randint(120, 124, (blocks, 1), generator=g).to(torch.uint8)
    bounds = dv.KeyBounds(hi_lo.cuda(), exp.cuda())
    table = torch.randperm(blocks, generator=g).int()
    q = torch.randn((1, 4, dim), generator=g).bfloat16()
    chunks = dv.Chunks(torch.tensor([0, 1]).int().cuda(), torch.tensor([blocks * page]).int().cuda(),
                       table[None].cuda().contiguous(), 1)
    got, status = dv.cache_select(cache, chunks, bounds, q.cuda(), 1000, 3, 4)
    torch.cuda.synchronize()
    x = q[0].double()
    n = (x / 2.0 ** least(float(x.abs().max()) * 4, 1016)).round()
    w = torch.stack((n.clamp_min(0).sum(0), n.clamp_max(0).sum(0)))
    score = ((hi_lo[table.long(), 0].double() * w).sum((1, 2)) * 2.0 ** (exp[table.long(), 0].double() - 127)).numpy()
    score[:3] = score[-4:] = math.inf
    want = np.sort(np.argsort(-score, kind="stable")[:1000])
    assert int(status.item()) == dv.OK and np.array_equal(got[0, 0].cpu().numpy(), want)


# ------------------------------------------------------------------ attention

def blocks64(st, q, scale, blocks):
    """(reference, tolerance) [rows, heads, dim]: see attention64 of the dense attention for the
    terms; 2^-8 A is the weights' rounding to bf16 (fp16 over e4m3 pages: less)."""
    heads = q.shape[1]
    g = heads // st.kv_heads
    q = f64(q)
    kh, vh = st.held()
    ref, tol = np.full(q.shape, math.nan), np.zeros(q.shape)
    for s in range(len(st.q)):
        k, v = st.tokens(kh, s), st.tokens(vh, s)
        for i in range(st.q[s]):
            r, p = st.off[s] + i, st.kv[s] - st.q[s] + i
            for h in range(heads):
                own = [b for b in blocks[r, h // g].tolist() if 0 <= b <= p // st.page] if p >= 0 else []
                j = np.array([x for b in own for x in range(b * st.page, min((b + 1) * st.page, p + 1))], dtype=int)
                if len(j) == 0:
                    ref[r, h] = 0
                    continue
                kk, vv = k[j, h // g], v[j, h // g]
                z = (kk @ q[r, h]) * scale
                w = np.exp(z - z.max())
                w /= w.sum()
                ref[r, h] = w @ vv
                big = (np.abs(kk) @ np.abs(q[r, h])).max() * scale
                tol[r, h] = (2.0 ** -8 * np.abs(ref[r, h])
                             + (w @ np.abs(vv)) * (2.0 ** -8 + 2.0 ** -12 + 2 * (st.dim + 2) * 2.0 ** -24 * big))
    return ref, tol


def random_lists(st, top, seed=0):
    """Lists in any order, with entries that name nothing and some twice."""
    r = np.random.default_rng(seed)
    out = np.full((st.rows, st.kv_heads, top), -1)
    for s in range(len(st.q)):
        for i in range(st.q[s]):
            own = max((st.kv[s] - st.q[s] + i) // st.page, 0)
            for h in range(st.kv_heads):
                out[st.off[s] + i, h] = r.integers(-1, own + 2, top)
    return torch.from_numpy(out).int()


def check_blocks(dv, st, heads, blocks, q=None, scale=None):
    q = st.queries(heads) if q is None else q
    scale = st.dim ** -0.5 if scale is None else scale
    out = torch.full((st.rows, heads, st.dim), 7.0, dtype=torch.bfloat16, device="cuda")
    got, status = dv.cache_attention_blocks(st.cache, st.chunks, q, blocks.cuda(), scale=scale, out=out)
    torch.cuda.synchronize()
    assert int(status.item()) == dv.OK
    ref, tol = blocks64(st, q, scale, blocks)
    got = f64(got)
    mine = np.zeros(st.rows, dtype=bool)
    mine[st.off[0]:st.off[-1]] = True
    assert (got[~mine] == 7.0).all()
    err = np.abs(got[mine] - ref[mine])
    bad = ~(err <= tol[mine])
    assert not bad.any(), (bad.sum(), np.nanmax(err / np.maximum(tol[mine], 1e-300)), np.argwhere(bad)[:4].tolist())
    return got


ATTEND = [
    # q, kv, kv_heads, dim, page, heads, top
    ([1], [1], 1, 64, 16, 1, 1),
    ([1], [700], 8, 128, 16, 40, 9),                   # one row: clusters
    ([1], [3000], 2, 128, 64, 16, 30),
    ([1, 1, 1], [17, 900, 333], 2, 64, 32, 10, 5),
    ([1] * 30, [37 * i + 1 for i in range(30)], 4, 128, 128, 28, 3),
    ([3, 0, 5], [200, 40, 5], 3, 128, 16, 3, 4),
    ([150], [150], 8, 64, 16, 64, 3),                  # a warp an item
    ([90, 33], [1000, 40], 10, 128, 64, 50, 2),
    ([20], [300], 1, 64, 16, 128, 7),                  # groups of 16 and more
    ([5], [400], 2, 128, 32, 18, 6),                   # nine heads: a group and a rest
    ([7], [400], 2, 128, 32, 40, 6),                   # twenty
    ([30], [25], 2, 64, 16, 4, 3),                     # front padding
    ([2], [5000], 1, 128, 16, 4, 200),
]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("case", range(len(ATTEND)))
def test_attention_over_blocks(dv, case, kind):
    q, kv, kv_heads, dim, page, heads, top = ATTEND[case]
    st = Setup(dv, q, kv, kv_heads, dim, page, kind, seed=case, front=1, back=3)
    check_blocks(dv, st, heads, random_lists(st, top, case))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_places_without_tokens_have_no_part_in_it(dv, kind, value):
    st = Setup(dv, [1, 4, 20], [30, 100, 77], 2, 128, 32, kind, fill=value)
    lists = torch.full((st.rows, 2, 5), -1).int()
    lists[..., :4] = torch.arange(4).int()
    check_blocks(dv, st, 10, lists)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_hidden_tokens_that_are_not_finite(dv, kind):
    """Later tokens of a row's own block, infinite or NaN, do not reach it; tokens that it sees do."""
    st = Setup(dv, [16], [16], 1, 64, 16, kind)
    p = int(st.table[0, 0])
    for t, e in ((st.cache.k, st.cache.k_exp), (st.cache.v, st.cache.v_exp)):
        if e is None:
            t[p, 0, 9, 3] = math.inf if t is st.cache.v else math.nan
        else:
            t[p, 0, 9] = 127
            e[p, 0, 9] = 255
    lists = torch.zeros((16, 1, 1)).int()
    q = st.queries(4)
    got, status = dv.cache_attention_blocks(st.cache, st.chunks, q, lists.cuda())
    torch.cuda.synchronize()
    assert int(status.item()) == dv.OK
    ref, tol = blocks64(st, q, 64 ** -0.5, lists)
    got = f64(got)
    assert (np.abs(got[:9] - ref[:9]) <= tol[:9]).all() and not np.isfinite(got[9:]).all(-1).any()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("rows", [1, 200])
def test_peaked_and_flat_scores(dv, kind, rows):
    """Scores that rise from tile to tile, by far, and ones that are all alike."""
    st = Setup(dv, [rows], [rows + 400], 1, 128, 16, kind, seed=4)
    lists = torch.arange(25).int().expand(rows, 1, 25).contiguous()
    check_blocks(dv, st, 5, lists, q=st.queries(5, scale=30.0))
    check_blocks(dv, st, 5, lists, q=torch.zeros((rows, 5, 128), dtype=torch.bfloat16, device="cuda"))
    check_blocks(dv, st, 5, lists, scale=3.0)


@pytest.mark.parametrize("rows", [1, 64])
def test_far_exponents(dv, rows):
    """e4m3: values whose exponents lie far apart from key to key, rows of zeros among them."""
    st = Setup(dv, [rows], [rows + 300], 2, 64, 16, "e4m3", seed=8)
    r = np.random.default_rng(2)
    e = r.choice([10, 40, 90, 127, 140], st.cache.v_exp.shape)
    st.cache.v_exp.copy_(torch.from_numpy(e.astype(np.uint8)))
    zero = torch.from_numpy(r.random(st.cache.v_exp.shape) < 0.2).cuda()
    st.cache.v.masked_fill_(zero[..., None], 0)
    st.cache.v_exp.masked_fill_(zero, 10)
    lists = torch.arange(18).int().expand(rows, 2, 18).contiguous()
    check_blocks(dv, st, 6, lists)
    st.cache.v_exp.fill_(240)
    st.cache.v.masked_fill_((st.cache.v & 127) > 112, 40)
    check_blocks(dv, st, 6, lists)
    st.cache.v.fill_(0)
    st.cache.v_exp.fill_(10)
    assert (check_blocks(dv, st, 6, lists) == 0).all()


def test_zeros_where_nothing_is_listed(dv):
    for kind in ("bf16", "e4m3"):
        st = Setup(dv, [2, 3], [100, 3], 2, 64, 16, kind)
        got = check_blocks(dv, st, 4, torch.full((5, 2, 3), -1).int())
        assert (got == 0).all()
        big = torch.tensor([7, 2 ** 31 - 1, -2 ** 31]).int().expand(5, 2, 3).contiguous()
        assert (check_blocks(dv, st, 4, big) == 0).all()


def test_pages_that_are_not_there(dv):
    st = Setup(dv, [1], [100], 1, 64, 16, "bf16")
    st.chunks.table[0, 2] = st.n_pages
    st.chunks.table[0, 3] = -1
    lists = torch.tensor([0, 2, 3, 6]).int().view(1, 1, 4)
    q = st.queries(2)
    got, status = dv.cache_attention_blocks(st.cache, st.chunks, q, lists.cuda())
    torch.cuda.synchronize()
    assert int(status.item()) == dv.ERANGE
    ref, tol = blocks64(st, q, 64 ** -0.5, torch.tensor([0, 6, -1, -1]).int().view(1, 1, 4))
    assert (np.abs(f64(got) - ref) <= tol).all()


def test_bad_sequences_are_left_out(dv):
    for rows in (1, 40):
        st = make(dv, [rows, rows, rows], [100, 100, 100], 2, 64, 16, "bf16", cols=9)
        good = st.chunks.kv_len.clone()
        lists = torch.arange(7).int().expand(3 * rows, 2, 7).contiguous().cuda()
        q = st.queries(4)
        want = dv.cache_attention_blocks(st.cache, st.chunks, q, lists)[0]
        chosen = dv.cache_select(st.cache, st.chunks, st.bounds, q, 5)[0]
        st.chunks.kv_len[1] = 9 * 16 + 1
        a, status = dv.cache_attention_blocks(st.cache, st.chunks, q, lists)
        b, status2 = dv.cache_select(st.cache, st.chunks, st.bounds, q, 5)
        status3 = dv.cache_bounds(st.cache, st.chunks, st.bounds, st.rows)
        torch.cuda.synchronize()
        assert [int(x.item()) for x in (status, status2, status3)] == [dv.ERANGE] * 3
        keep = list(range(rows)) + list(range(2 * rows, 3 * rows))
        assert torch.equal(a[keep], want[keep]) and torch.equal(b[keep], chosen[keep])
        st.chunks.kv_len.copy_(good)


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_all_blocks_are_the_dense_attention(dv, kind):
    """Lists of every block give what the dense attention gives, within both tolerances."""
    st = make(dv, [1, 60, 9], [333, 200, 9], 4, 128, 16, kind)
    q = st.queries(20)
    blocks, status = dv.cache_select(st.cache, st.chunks, st.bounds, q, 21, 1, 1)
    check_blocks(dv, st, 20, blocks.cpu(), q=q)
    check_attention(dv, st, 20, q=q)
    assert int(status.item()) == dv.OK


def test_the_same_bits_again_and_on_another_stream(dv):
    st = make(dv, [1, 130], [5000, 3000], 8, 128, 64, "e4m3")
    q = st.queries(40)
    first = None
    for _ in range(20):
        blocks, _ = dv.cache_select(st.cache, st.chunks, st.bounds, q, 9, 1, 2)
        out, _ = dv.cache_attention_blocks(st.cache, st.chunks, q, blocks)
        if first is None:
            first = blocks, out
        assert torch.equal(first[0], blocks) and torch.equal(first[1], out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        blocks, _ = dv.cache_select(st.cache, st.chunks, st.bounds, q, 9, 1, 2)
        out, _ = dv.cache_attention_blocks(st.cache, st.chunks, q, blocks)
    s.synchronize()
    assert torch.equal(first[0], blocks) and torch.equal(first[1], out)


def test_a_long_prompt_and_its_answer(dv):
    """Projection rows -> norm and rotation -> pages -> cache -> bounds -> selection -> attention, a prompt in
    chunks and then a captured step of single tokens whose sequences are forked in between."""
    torch.manual_seed(0)
    heads, hk, dim, page, top = 10, 2, 64, 16, 6
    pool, tables = dv.PagePool.empty(200, page), dv.PageTables.empty(8, 40)
    copies = dv.PageCopies(200)
    cache = dv.KvCache.empty(200, hk, page, dim)
    bounds = dv.KeyBounds.empty(cache)
    rotary = dv.Rotary(dim, 10000.0, (12, 10, 10), True)
    weights = [(1 + 0.1 * torch.randn(dim)).bfloat16().cuda() for _ in range(2)]
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")   # noqa: E731
    history = {0: ([], [])}          # slot -> what its cache holds: keys, values

    def step(slots, new, qkv, ch):
        rows = sum(new)
        x = qkv.view(rows, heads + 2 * hk, dim)
        q, k, v = x[:, :heads], x[:, heads:heads + hk], x[:, heads + hk:]
        lens = [len(history[s][0]) for s in slots]
        pos = torch.cat([torch.arange(l, l + c) for l, c in zip(lens, new)]).int().expand(3, rows).contiguous().cuda()
        q, k = dv.qk_norm_rope(rotary, q, k, pos, *weights)
        dv.cache_write(cache, ch, k, v, status)
        dv.cache_bounds(cache, ch, bounds, rows, status)
        blocks, _ = dv.cache_select(cache, ch, bounds, q, top, 1, 2, status=status)
        out, _ = dv.cache_attention_blocks(cache, ch, q, blocks, status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == dv.OK
        at = 0
        for s, c, l in zip(slots, new, lens):
            for i in range(c):
                history[s][0].append(f64(k[at + i]))
                history[s][1].append(f64(v[at + i]))
            for i in range(c):
                p, r = l + i, at + i
                ks, vs = np.array(history[s][0]), np.array(history[s][1])
                for h in range(heads):
                    own = [b for b in blocks[r, h // 5].tolist() if b >= 0]
                    assert own[0] == 0 and own[-1] == p // page and len(own) == min(top, p // page + 1)
                    j = np.array([x for b in own for x in range(b * page, min(p + 1, b * page + page))])
                    z = ks[j, h // 5] @ f64(q[r, h]) / 8
                    w = np.exp(z - z.max())
                    w /= w.sum()
                    err = np.abs(f64(out[r, h]) - w @ vs[j, h // 5])
                    assert (err <= 2.0 ** -8 * np.abs(w @ vs[j, h // 5]) + 1.2 * 2.0 ** -8 * (w @ np.abs(vs[j, h // 5]))).all()
            at += c

    def chunks(slots, new):
        off = np.concatenate([[0], np.cumsum(new)]).tolist()
        at = torch.tensor(slots, device="cuda")
        return dv.Chunks(i32(off), tables.kv_len[at].contiguous(), tables.table[at].contiguous(), max(new))

    for c in (100, 53, 90):
        dv.pages_resize(pool, tables, i32([0]), i32([len(history[0][0]) + c]), copies, status)
        step([0], [c], torch.randn(c, (heads + 2 * hk) * dim).bfloat16().cuda(), chunks([0], [c]))
    dv.pages_fork(pool, tables, i32([0, 0]), i32([1, 2]), copies, status)
    dv.cache_copy(cache, copies, bounds, status)
    for s in (1, 2):
        history[s] = (list(history[0][0]), list(history[0][1]))
    for turn in range(20):
        n = len(history[0][0]) + 1
        dv.pages_resize(pool, tables, i32([0, 1, 2]), i32([n, n, n]), copies, status)
        if turn == 9:
            dv.pages_compact(pool, tables, copies, status)
            dv.cache_copy(cache, copies, bounds, status)
        step([0, 1, 2], [1, 1, 1], torch.randn(3, (heads + 2 * hk) * dim).bfloat16().cuda(), chunks([0, 1, 2], [1, 1, 1]))


def test_captured_step(dv):
    """Bounds, selection and attention in one graph; replays read lengths, tables and queries anew."""
    st = make(dv, [1, 1, 1], [200, 333, 64], 4, 128, 16, "bf16", cols=30)
    q = st.queries(20).contiguous()
    blocks = torch.zeros((3, 4, 7), dtype=torch.int32, device="cuda")
    out = torch.zeros((3, 20, 128), dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def step():
        dv.cache_bounds(st.cache, st.chunks, st.bounds, 3, status)
        dv.cache_select(st.cache, st.chunks, st.bounds, q, 7, 1, 2, out=blocks, status=status)
        dv.cache_attention_blocks(st.cache, st.chunks, q, blocks, out=out, status=status)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for lens in ([200, 333, 64], [100, 17, 1], [1, 320, 40]):
        st.chunks.kv_len.copy_(torch.tensor(lens))
        q.neg_()
        graph.replay()
        got = blocks.clone(), out.clone()
        blocks.zero_()
        out.zero_()
        step()
        torch.cuda.synchronize()
        assert torch.equal(got[0], blocks) and torch.equal(got[1], out) and int(status.item()) == dv.OK


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_rows_that_are_parts_of_wider_ones(dv, kind):
    """Queries out of a projection's rows, outputs into wider ones: the same, and what lies beside stays."""
    st = make(dv, [1, 77, 3], [400, 300, 90], 4, 128, 16, kind, back=2)
    q = st.queries(20, wide=8)
    assert q.stride(0) == 28 * 128
    blocks, _ = dv.cache_select(st.cache, st.chunks, st.bounds, q.contiguous(), 6, 1, 1)
    want, _ = dv.cache_attention_blocks(st.cache, st.chunks, q.contiguous(), blocks)
    wide = torch.full((st.rows, 23, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    got, _ = dv.cache_select(st.cache, st.chunks, st.bounds, q, 6, 1, 1)
    out, status = dv.cache_attention_blocks(st.cache, st.chunks, q, blocks, out=wide[:, 2:22])
    torch.cuda.synchronize()
    n = st.off[-1]
    assert int(status.item()) == dv.OK and torch.equal(got[:n], blocks[:n]) and torch.equal(out[:n], want[:n])
    assert (wide[:, :2] == 3).all() and (wide[:, 22:] == 3).all() and (wide[n:] == 3).all()


def test_two_streams_at_once(dv):
    sts = [make(dv, [1, 100], [3000, 2000], 8, 128, 16, kind, seed=i) for i, kind in enumerate(("bf16", "e4m3"))]
    qs = [st.queries(40) for st in sts]

    def step(st, q):
        dv.cache_bounds(st.cache, st.chunks, st.bounds, st.rows)
        blocks, _ = dv.cache_select(st.cache, st.chunks, st.bounds, q, 20, 1, 2)
        return blocks, dv.cache_attention_blocks(st.cache, st.chunks, q, blocks)[0]

    want = [step(st, q) for st, q in zip(sts, qs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sts]
    got = [[], []]
    for _ in range(15):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(step(sts[i], qs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for blocks, out in got[i]:
            assert torch.equal(blocks, want[i][0]) and torch.equal(out, want[i][1])


def test_lists_laid_out_otherwise(dv):
    """Heads in front of rows, and room between the lists."""
    st = make(dv, [1, 130], [500, 300], 4, 64, 16, "bf16")
    q = st.queries(20)
    blocks, _ = dv.cache_select(st.cache, st.chunks, st.bounds, q, 9, 1, 2)
    out, _ = dv.cache_attention_blocks(st.cache, st.chunks, q, blocks)
    wide = torch.full((4, st.rows, 13), 99, dtype=torch.int32, device="cuda")
    lists = wide.transpose(0, 1)[..., 2:11]
    got, _ = dv.cache_select(st.cache, st.chunks, st.bounds, q, 9, 1, 2, out=lists)
    again, status = dv.cache_attention_blocks(st.cache, st.chunks, q, lists)
    torch.cuda.synchronize()
    assert int(status.item()) == dv.OK and torch.equal(lists, blocks) and torch.equal(again, out)
    assert (wide[..., :2] == 99).all() and (wide[..., 11:] == 99).all()
    with pytest.raises(dv.DsVitError):
        dv.cache_attention_blocks(st.cache, st.chunks, q, blocks.transpose(1, 2).contiguous().transpose(1, 2))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_a_cache_past_32_bits(dv, kind):
    """Pages whose bytes, and whose values, lie past 2^32: the same as at the front of the cache."""
    heads, page, dim, used = 8, 64, 128, 9
    n = 34000 if kind == "bf16" else 67000
    cache = dv.KvCache.empty(n, heads, page, dim, dv.CACHE_BF16 if kind == "bf16" else dv.CACHE_E4M3)
    assert cache.k.numel() * cache.k.element_size() > 2 ** 32
    for t in (cache.k, cache.v):
        if kind == "bf16":
            t[:used].copy_(torch.randn(t[:used].shape, device="cuda"))
        else:
            t[:used].copy_(torch.randint(0, 120, t[:used].shape, device="cuda"))
    if kind == "e4m3":
        for e in (cache.k_exp, cache.v_exp):
            e[:used].copy_(torch.randint(118, 124, e[:used].shape, device="cuda"))
    copies = dv.PageCopies(used)
    copies.src.copy_(torch.arange(used))
    copies.dst.copy_(torch.arange(n - used, n))
    copies.count.fill_(used)
    bounds = dv.KeyBounds.empty(cache)
    q = torch.randn((40, 40, dim), device="cuda").bfloat16()
    got = []
    for rows, kv in ((1, used * page), (40, used * page - 5)):
        for first in (0, n - used):
            table = torch.arange(first, first + used, device="cuda").int()[None].contiguous()
            ch = dv.Chunks(torch.tensor([0, rows]).int().cuda(), torch.tensor([kv]).int().cuda(), table, rows)
            whole = dv.Chunks(torch.tensor([0, kv]).int().cuda(), torch.tensor([kv]).int().cuda(), table, kv)
            status = dv.cache_copy(cache, copies)
            dv.cache_bounds(cache, whole, bounds, kv, status)
            blocks, _ = dv.cache_select(cache, ch, bounds, q[:rows], 5, 1, 1, status=status)
            out, _ = dv.cache_attention_blocks(cache, ch, q[:rows], blocks, status=status)
            torch.cuda.synchronize()
            assert int(status.item()) == dv.OK
            got.append((blocks, out))
        assert torch.equal(got[-1][0], got[-2][0]) and torch.equal(got[-1][1], got[-2][1])
        assert torch.isfinite(got[-1][1]).all() and (got[-1][1] != 0).any()


def test_no_rows(dv):
    st = make(dv, [1], [20], 2, 64, 16, "bf16")
    q = torch.zeros((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    blocks, status = dv.cache_select(st.cache, st.chunks, st.bounds, q, 3)
    assert blocks.shape == (0, 2, 3)
    assert dv.cache_attention_blocks(st.cache, st.chunks, q, blocks)[0].shape == (0, 4, 64)
    dv.cache_bounds(st.cache, st.chunks, st.bounds, 0, status)
    torch.cuda.synchronize()
    assert int(status.item()) == dv.OK

"""The paged K/V cache on the GPU: writing, reading back and attention against
plain implementations in 64 bits, their masks, paddings and refusals, and a
prompt taken through them as a serving loop would."""
import math

import numpy as np
import pytest

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


# ------------------------------------------------------------------ a plain model of the cache

def e4m3_values():
    """The 256 values of the format: sign, 4 exponent bits (bias 7), 3 mantissa bits."""
    out = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = math.nan if (b & 127) == 127 else (m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
        out[b] = -x if b & 128 else x
    return out


E4M3 = e4m3_values()


def quantise(x):
    """Rows [..., d] of float64 -> (bytes, exponent bytes), by the definition: the
    nearest value of the format, the one with the even last bit on a tie."""
    x = np.asarray(x, dtype=np.float64)
    a = np.abs(x).max(-1)
    fine = np.isfinite(a)
    e = np.full(a.shape, -117)
    for cand in range(121, -118, -1):              # the least e with a <= 448 2^e
        e = np.where(fine & (a <= 448 * 2.0 ** cand), cand, e)
    scaled = np.where(fine[..., None], np.abs(x), 0) / 2.0 ** e[..., None]
    pos = E4M3[:127]
    hi = np.searchsorted(pos, scaled).clip(0, 126)
    lo = (hi - 1).clip(0)
    dl, dh = scaled - pos[lo], pos[hi] - scaled
    pick = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    pick = np.where(e[..., None] == 120, np.minimum(pick, 119), pick)     # at most 240 2^120: finite in bf16
    bits = np.where(fine[..., None], pick | (np.signbit(x) * 128), 127)
    return bits.astype(np.uint8), np.where(fine, e + 127, 255).astype(np.uint8)


def f64(t):
    return t.detach().cpu().double().numpy()


class Setup:
    """Sequences of q[s] new rows and kv[s] cached tokens; a random page table;
    front / back extra packed rows that belong to no sequence."""

    def __init__(self, dv, q, kv, kv_heads, dim, page, kind, seed=0, front=0, back=0, cols=None, max_rows=None,
                 fill=None):
        g = torch.Generator().manual_seed(seed)
        self.q, self.kv, self.kv_heads, self.dim, self.page, self.kind = q, kv, kv_heads, dim, page, kind
        n = len(q)
        used = [-(-x // page) for x in kv]
        self.n_pages = sum(used) + 2
        cols = max(max(used), 1) if cols is None else cols
        order = torch.randperm(self.n_pages, generator=g).int()
        self.spare = int(order[-1])
        self.table = torch.full((n, cols), -1, dtype=torch.int32)
        at = 0
        for s, u in enumerate(used):
            self.table[s, :u] = order[at:at + u]
            at += u
        self.off = [front + sum(q[:s]) for s in range(n + 1)]
        self.rows = self.off[-1] + back
        self.chunks = dv.Chunks(torch.tensor(self.off, dtype=torch.int32).cuda(),
                                torch.tensor(kv, dtype=torch.int32).cuda(), self.table.cuda(),
                                max(max(q), 1) if max_rows is None else max_rows)
        shape = (self.n_pages, kv_heads, page, dim)
        if kind == "bf16":
            k, v = (torch.randn(shape, generator=g) for _ in range(2))
            k = k * torch.exp(0.5 * torch.randn((kv_heads, 1, dim), generator=g))
            self.cache = dv.KvCache(k.bfloat16().cuda(), v.bfloat16().cuda())
        else:
            parts = []
            for _ in range(2):
                b, e = quantise(torch.randn(shape, generator=g).bfloat16().double().numpy()
                                * 2.0 ** torch.randint(-3, 3, shape[:3] + (1,), generator=g).numpy())
                parts.append((torch.from_numpy(b).cuda(), torch.from_numpy(e).cuda()))
            self.cache = dv.KvCache(parts[0][0], parts[1][0], parts[0][1], parts[1][1])
        self.g = g
        if fill is not None:
            self.spoil(fill)

    def spoil(self, value):
        """`value` in every slot that holds no token: whole spare pages and the ends of last pages."""
        free = torch.ones((self.n_pages, self.page), dtype=torch.bool)
        for s, x in enumerate(self.kv):
            for j in range(x):
                free[int(self.table[s, j // self.page]), j % self.page] = False
        free = free.cuda()[:, None, :]
        for t, e in ((self.cache.k, self.cache.k_exp), (self.cache.v, self.cache.v_exp)):
            if e is None:
                t.masked_fill_(free[..., None], value)
            else:
                t.masked_fill_(free[..., None], 127)
                e.masked_fill_(free, 255)

    def held(self):
        """(k, v) float64 [n_pages, kv_heads, page, dim]: what the pages stand for."""
        out = []
        for t, e in ((self.cache.k, self.cache.k_exp), (self.cache.v, self.cache.v_exp)):
            if e is None:
                out.append(f64(t))
            else:
                ex = e.cpu().numpy().astype(np.int64)
                x = E4M3[t.cpu().numpy()] * 2.0 ** (ex[..., None] - 127.0)
                out.append(np.where(ex[..., None] == 255, math.nan, x))
        return out

    def tokens(self, held, s):
        """[kv, kv_heads, dim] of sequence s in order."""
        j = np.arange(self.kv[s])
        return held[self.table[s].numpy()[j // self.page], :, j % self.page].reshape(-1, self.kv_heads, self.dim)

    def queries(self, heads, scale=1.0, wide=0):
        x = torch.randn((self.rows, heads + wide, self.dim), generator=self.g) * scale
        return x.bfloat16().cuda()[:, :heads]


def attention64(st, q, scale, window=0, sinks=0):
    """(reference, tolerance) [rows, heads, dim] in 64 bits, NaN rows for rows
    outside every sequence.

    Tolerance of one output o = sum_j w_j v_j (w the softmax weights): the result
    is rounded to bf16 (2^-8 |o|); each weight is rounded to bf16 before its
    product (2^-8 A, A = sum_j w_j |v_j|); fp32 scores carry up to (dim + 2)
    2^-24 sum_d |q_d k_d| each, in the weight and in their sum (twice that,
    relative to A); exponentials, sums and rescalings in fp32 stay under 2^-12 A.
    """
    heads = q.shape[1]
    g = heads // st.kv_heads
    q = f64(q)
    kh, vh = st.held()
    ref = np.full(q.shape, math.nan)
    tol = np.zeros(q.shape)
    for s in range(len(st.q)):
        k, v = st.tokens(kh, s), st.tokens(vh, s)
        c = st.q[s]
        for i in range(c):
            r, p = st.off[s] + i, st.kv[s] - c + i
            j = np.arange(p + 1)
            if window:
                j = j[(j > p - window) | (j < sinks)]
            if len(j) == 0:
                ref[r] = 0
                continue
            for h in range(heads):
                kk, vv = k[j, h // g], v[j, h // g]
                z = (kk @ q[r, h]) * scale
                w = np.exp(z - z.max())
                w /= w.sum()
                ref[r, h] = w @ vv
                big = (np.abs(kk) @ np.abs(q[r, h])).max() * scale
                tol[r, h] = (2.0 ** -8 * np.abs(ref[r, h])
                             + (w @ np.abs(vv)) * (2.0 ** -8 + 2.0 ** -12 + 2 * (st.dim + 2) * 2.0 ** -24 * big))
    return ref, tol


def check_attention(dv, st, heads, window=0, sinks=0, q=None, scale=None):
    q = st.queries(heads) if q is None else q
    scale = st.dim ** -0.5 if scale is None else scale
    out = torch.full((st.rows, heads, st.dim), 7.0, dtype=torch.bfloat16, device="cuda")
    got, status = dv.cache_attention(st.cache, st.chunks, q, scale=scale, window=window, sinks=sinks, out=out)
    torch.cuda.synchronize()
    assert int(status.item()) == dv.OK
    ref, tol = attention64(st, q, scale, window, sinks)
    got = f64(got)
    mine = np.zeros(st.rows, dtype=bool)
    mine[st.off[0]:st.off[-1]] = True
    assert (got[~mine] == 7.0).all()                       # rows of no sequence stay as they were
    err = np.abs(got[mine] - ref[mine])
    bad = ~(err <= tol[mine])
    assert not bad.any(), (f"{bad.sum()} of {bad.size} outside, worst "
                           f"{np.nanmax(err / np.maximum(tol[mine], 1e-30))} times the tolerance at "
                           f"{np.argwhere(bad)[:4].tolist()}")
    return got


# ------------------------------------------------------------------ writing and reading

WRITE_CASES = [
    # q, kv, kv_heads, dim, page, kind, front, back
    ([1], [1], 1, 64, 16, "bf16", 0, 0),
    ([1], [16], 1, 128, 16, "e4m3", 0, 0),
    ([1, 1, 1, 1, 1], [1, 17, 32, 33, 500], 8, 128, 32, "bf16", 0, 3),
    ([3, 0, 40, 1], [3, 100, 57, 64], 2, 64, 16, "e4m3", 2, 5),
    ([130, 7, 300], [130, 20, 555], 3, 128, 64, "e4m3", 0, 1),
    ([200, 0, 0, 129], [200, 0, 5, 1000], 5, 64, 128, "bf16", 4, 0),
    ([9, 5], [4, 0], 4, 128, 16, "e4m3", 1, 1),            # rows in front of position 0
    ([2] * 300, [2 + i for i in range(300)], 2, 64, 32, "bf16", 0, 0),
    ([1, 0] * 512, [1 + i % 70 for i in range(1024)], 1, 64, 16, "e4m3", 0, 0),
    ([33], [33], 10, 128, 16, "bf16", 0, 0),
]


@pytest.mark.parametrize("q,kv,kv_heads,dim,page,kind,front,back", WRITE_CASES)
def test_write_and_read(dv, q, kv, kv_heads, dim, page, kind, front, back):
    """Every byte of the pages after a write, and every row read back, equal the
    definition's; slots without a new token keep their bytes."""
    st = Setup(dv, q, kv, kv_heads, dim, page, kind, seed=len(q) + dim, front=front, back=back)
    x = torch.randn((st.rows, 2 * kv_heads + 1, dim), generator=st.g) * torch.exp(
        2 * torch.randn((st.rows, 2 * kv_heads + 1, 1), generator=st.g))
    x = x.bfloat16().cuda()
    k, v = x[:, 1:1 + kv_heads], x[:, 1 + kv_heads:]        # rows inside a wider tensor
    want = []
    for t, e, new in ((st.cache.k, st.cache.k_exp, k), (st.cache.v, st.cache.v_exp, v)):
        bits = (t.view(torch.int16) if kind == "bf16" else t).cpu().numpy().copy()
        ex = None if e is None else e.cpu().numpy().copy()
        rows = new.contiguous().cpu()
        nb, ne = (rows.view(torch.int16).numpy(), None) if kind == "bf16" else quantise(rows.double().numpy())
        for s in range(len(q)):
            for i in range(q[s]):
                p = kv[s] - q[s] + i
                if p < 0:
                    continue
                page_no, slot = int(st.table[s, p // page]), p % page
                bits[page_no, :, slot] = nb[st.off[s] + i]
                if ne is not None:
                    ex[page_no, :, slot] = ne[st.off[s] + i]
        want.append((bits, ex))
    status = dv.cache_write(st.cache, st.chunks, k, v)
    torch.cuda.synchronize()
    assert int(status.item()) == dv.OK
    for (bits, ex), t, e in zip(want, (st.cache.k, st.cache.v), (st.cache.k_exp, st.cache.v_exp)):
        assert np.array_equal((t.view(torch.int16) if kind == "bf16" else t).cpu().numpy(), bits)
        assert e is None or np.array_equal(e.cpu().numpy(), ex)
    wide = torch.full((st.rows, 2 * kv_heads + 1, dim), 7.0, dtype=torch.bfloat16, device="cuda")
    rk, rv, status = dv.cache_read(st.cache, st.chunks, st.rows, out=(wide[:, :kv_heads], wide[:, kv_heads + 1:]))
    torch.cuda.synchronize()
    assert int(status.item()) == dv.OK
    assert bool((wide[:, kv_heads] == 7.0).all())
    for got, held in zip((rk, rv), st.held()):
        got = f64(got)
        assert (got[:st.off[0]] == 7.0).all() and (got[st.off[-1]:] == 7.0).all()
        for s in range(len(q)):
            ref = np.zeros((q[s], kv_heads, dim))
            t = min(q[s], kv[s])
            if t:
                ref[q[s] - t:] = st.tokens(held, s)[kv[s] - t:]
            assert np.array_equal(got[st.off[s]:st.off[s + 1]], ref)


MANY_ROWS = [
    # More rows than run at once and few heads: several tokens a warp.
    ([9000, 3000], [9000, 3500], 1, 128, 64, "e4m3", 0, 0),
    ([11000], [11001], 1, 64, 16, "bf16", 3, 7),
    ([20] * 600, [20 + i % 50 for i in range(600)], 2, 64, 32, "e4m3", 5, 1),
    ([17, 0, 40, 1] * 250, [9, 3, 57, 64] * 250, 3, 64, 128, "bf16", 1, 200),    # rows in front of position 0
    ([5000, 0, 4999], [5000, 0, 6000], 4, 128, 32, "e4m3", 0, 40),
    ([10007], [10007], 7, 64, 16, "e4m3", 2, 2),
]


@pytest.mark.parametrize("q,kv,kv_heads,dim,page,kind,front,back", MANY_ROWS)
def test_write_and_read_of_many_rows(dv, q, kv, kv_heads, dim, page, kind, front, back):
    test_write_and_read(dv, q, kv, kv_heads, dim, page, kind, front, back)


def test_write_e4m3_special_values(dv):
    """Zeros, every bf16 magnitude as a row's largest, ties, values far below the
    largest, infinities and NaN."""
    n = 32768
    st = Setup(dv, [n], [n], 1, 64, 128, "e4m3", seed=3)
    bits = torch.arange(n, dtype=torch.int32).to(torch.int16)
    x = torch.zeros((n, 64), dtype=torch.int16)
    x[:, 5] = bits
    x[:, 6] = torch.where(bits > 128 * 20, bits - 128 * 17, torch.zeros_like(bits)) | -32768
    x[:, 7] = torch.where(bits > 128 * 8, bits - 128 * 3 + 1, torch.zeros_like(bits))
    x[:, 63] = torch.where(bits > 128 * 10, (bits & -128) - 128 * 9 + 24, torch.zeros_like(bits))
    k = x.view(torch.bfloat16).view(n, 1, 64)
    v = torch.flip(k, (0,)).contiguous()
    dv.cache_write(st.cache, st.chunks, k.cuda(), v.cuda())
    rk, rv, _ = dv.cache_read(st.cache, st.chunks, n)
    torch.cuda.synchronize()
    for src, t, e, back in ((k, st.cache.k, st.cache.k_exp, rk), (v, st.cache.v, st.cache.v_exp, rv)):
        wb, we = quantise(src.double().numpy())
        slots = st.table[0].numpy()[np.arange(n) // 128], np.arange(n) % 128
        gb, ge = t.cpu().numpy()[slots[0], :, slots[1]], e.cpu().numpy()[slots[0], :, slots[1]]
        assert np.array_equal(ge, we)
        assert np.array_equal(gb, wb)
        ref = np.where(we[..., None] == 255, math.nan, E4M3[wb] * 2.0 ** (we[..., None].astype(float) - 127))
        assert np.array_equal(f64(back), ref, equal_nan=True)
        fine = np.isfinite(src.double().numpy()).all(-1)
        # what is read back is off by at most half a step of the format: 2^-4 of
        # the value, or 2^-10 2^e where the scaled value is subnormal
        err = np.abs(f64(back) - src.double().numpy())[fine]
        step = 2.0 ** (we.astype(float)[..., None] - 127)[fine]
        assert (err <= np.maximum(2.0 ** -4 * np.abs(src.double().numpy()[fine]), 2.0 ** -10 * step)).all()


def test_read_every_byte(dv):
    """Every element byte under every exponent byte that a write can leave; at the
    largest exponent, elements above 240 (which a write does not leave there)
    stand for more than bf16 holds and read as infinities."""
    st = Setup(dv, [240], [240], 4, 64, 16, "e4m3", seed=1)
    every = torch.arange(256, dtype=torch.uint8)
    every[127], every[255] = 0, 128
    for t, e in ((st.cache.k, st.cache.k_exp), (st.cache.v, st.cache.v_exp)):
        t.copy_(every.view(1, 4, 1, 64).expand(t.shape))
        e.copy_((torch.arange(e.numel(), dtype=torch.int64) % 238 + 10).to(torch.uint8).view(e.shape))
    rk, rv, _ = dv.cache_read(st.cache, st.chunks, 240)
    torch.cuda.synchronize()
    for got, held in zip((rk, rv), st.held()):
        want = st.tokens(held, 0)
        want = np.where(np.abs(want) >= 2.0 ** 128, np.copysign(math.inf, want), want)
        assert np.array_equal(f64(got), want)


# ------------------------------------------------------------------ attention

ATTENTION_CASES = [
    # q, kv, heads, kv_heads, dim, page, kind
    ([1], [1], 1, 1, 64, 16, "bf16"),
    ([1], [2], 8, 8, 128, 16, "e4m3"),
    ([1], [129], 5, 1, 128, 16, "bf16"),
    ([1], [1000], 40, 8, 128, 64, "bf16"),
    ([1], [1000], 40, 8, 128, 64, "e4m3"),
    ([1] * 9, [1, 16, 17, 63, 64, 65, 300, 0, 777], 8, 2, 64, 32, "bf16"),
    ([1] * 9, [1, 16, 17, 63, 64, 65, 300, 0, 777], 14, 2, 128, 128, "e4m3"),
    ([1] * 70, [1 + 7 * i for i in range(70)], 4, 4, 64, 16, "e4m3"),
    ([4, 1, 0, 3], [4, 50, 9, 260], 16, 2, 128, 32, "bf16"),          # a few rows each
    ([5, 2, 6], [300, 2, 70], 7, 1, 64, 16, "e4m3"),
    ([2, 1], [90, 131], 32, 1, 128, 64, "bf16"),                       # 32 query heads on one
    ([1, 2], [40, 200], 128, 1, 64, 16, "bf16"),                       # the largest group
    ([17], [17], 2, 2, 64, 16, "bf16"),
    ([50], [400], 8, 8, 128, 16, "bf16"),                              # chunks
    ([65], [65], 10, 2, 128, 64, "e4m3"),
    ([128], [128], 2, 1, 64, 128, "bf16"),
    ([129, 3], [129, 513], 4, 1, 128, 32, "bf16"),
    ([100, 0, 260], [100, 7, 300], 6, 2, 64, 16, "e4m3"),
    ([130, 61], [700, 61], 5, 1, 128, 16, "e4m3"),                     # 5 heads a group: 125 of 128 rows
    ([90], [250], 21, 3, 64, 64, "bf16"),                              # 7 heads a group
    ([40], [170], 33, 1, 64, 32, "e4m3"),
    ([300], [1500], 4, 4, 128, 128, "bf16"),
    ([3], [40], 128, 1, 128, 16, "e4m3"),
]


@pytest.mark.parametrize("q,kv,heads,kv_heads,dim,page,kind", ATTENTION_CASES)
def test_attention(dv, q, kv, heads, kv_heads, dim, page, kind):
    st = Setup(dv, q, kv, kv_heads, dim, page, kind, seed=sum(q) + dim, fill=math.nan)
    check_attention(dv, st, heads)


MASKS = [(1, 0), (1, 1), (2, 3), (16, 4), (17, 0), (64, 1), (100, 37), (128, 128), (129, 5), (1000, 4), (10 ** 9, 0),
         (2 ** 31 - 1, 2 ** 31 - 1), (0, 7)]


@pytest.mark.parametrize("window,sinks", MASKS)
@pytest.mark.parametrize("q,kv,heads,kv_heads,dim,page,kind", [
    ([1, 1, 1], [700, 33, 1], 6, 2, 128, 16, "bf16"),
    ([3, 1], [520, 130], 8, 2, 64, 32, "e4m3"),
    ([70, 20], [500, 20], 4, 1, 128, 64, "e4m3"),
    ([200], [430], 2, 2, 64, 16, "bf16"),
])
def test_attention_window_and_sinks(dv, q, kv, heads, kv_heads, dim, page, kind, window, sinks):
    """Pages that no row's window reaches are given away: their table entries name
    no page, and nothing reads them."""
    st = Setup(dv, q, kv, kv_heads, dim, page, kind, seed=window % 97 + dim, fill=math.nan)
    check_attention(dv, st, heads, window, sinks, q=st.queries(heads))
    if window:
        away = st.chunks.table.clone()
        for s in range(len(q)):
            first = max(0, kv[s] - q[s] - window + 1)
            for c in range(away.shape[1]):
                if c * page >= sinks and (c + 1) * page <= first:
                    away[s, c] = -1
        st.chunks.table.copy_(away)
        check_attention(dv, st, heads, window, sinks, q=st.queries(heads))


@pytest.mark.parametrize("heads,kv_heads,dim,kind", [(4, 1, 128, "bf16"), (3, 3, 64, "e4m3"), (40, 8, 128, "e4m3")])
def test_attention_front_padding(dv, heads, kv_heads, dim, kind):
    """Rows in front of position 0 see nothing and give zeros, with rows of no
    sequence around them."""
    st = Setup(dv, [9, 5, 1, 70], [4, 0, 0, 30], kv_heads, dim, 16, kind, seed=5, front=3, back=6)
    got = check_attention(dv, st, heads)
    assert (got[3:8] == 0).all() and (got[12:18] == 0).all()


@pytest.mark.parametrize("scale", [1.0, 6.0])
@pytest.mark.parametrize("q,kv,heads,kv_heads,dim,kind", [
    ([1], [600], 8, 1, 128, "bf16"), ([1], [600], 8, 1, 64, "e4m3"),
    ([90], [600], 2, 1, 128, "bf16"), ([90], [600], 2, 1, 64, "e4m3")])
def test_attention_large_scores(dv, q, kv, heads, kv_heads, dim, kind, scale):
    """Scores of a hundred and more: the running maximum rises and stays right."""
    st = Setup(dv, q, kv, kv_heads, dim, 32, kind, seed=8)
    check_attention(dv, st, heads, q=st.queries(heads, 3.0), scale=scale * dim ** -0.5)


def _plant(st, s, j, head, value, what):
    """`value` into one element of token j's row (e4m3: the whole row becomes NaN)."""
    page, slot = int(st.table[s, j // st.page]), j % st.page
    t, e = (st.cache.k, st.cache.k_exp) if what == "k" else (st.cache.v, st.cache.v_exp)
    if e is None:
        t[page, head, slot, 3] = value
    else:
        t[page, head, slot] = 127
        e[page, head, slot] = 255


@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("q,kv,kind,dim,window,sinks", [
    ([4, 1], [200, 90], "bf16", 128, 0, 0), ([4, 1], [200, 90], "e4m3", 64, 0, 0),
    ([70, 3], [300, 70], "bf16", 64, 0, 0), ([70, 3], [300, 70], "e4m3", 128, 0, 0),
    ([70, 3], [300, 70], "bf16", 128, 30, 2), ([6, 2], [300, 70], "e4m3", 128, 30, 2),
])
def test_attention_hidden_values_have_no_part(dv, q, kv, kind, dim, window, sinks, value, what):
    """An infinity or NaN in a key or value that a row does not see leaves that
    row's result untouched; one that it sees gives NaN or the infinity."""
    st = Setup(dv, q, kv, 2, dim, 16, kind, seed=6)
    heads = 4
    query = st.queries(heads)
    clean, _ = dv.cache_attention(st.cache, st.chunks, query, window=window, sinks=sinks)
    clean = f64(clean)
    bad = kv[0] - q[0] + q[0] // 2            # a new token in the middle of the chunk
    _plant(st, 0, bad, 1, value, what)
    got, status = dv.cache_attention(st.cache, st.chunks, query, window=window, sinks=sinks)
    torch.cuda.synchronize()
    assert int(status.item()) == dv.OK
    got = f64(got)
    ref, tol = attention64(st, query, dim ** -0.5, window, sinks)
    for i in range(q[0]):
        p = kv[0] - q[0] + i
        seen = bad <= p and (window == 0 or bad > p - window or bad < sinks)
        assert np.array_equal(got[i, :2], clean[i, :2])                 # the other K/V head
        if not seen:
            assert (np.abs(got[i, 2:] - clean[i, 2:]) <= 2 * tol[i, 2:]).all(), i
        elif what == "v" and kind == "bf16":
            assert (np.isnan(got[i, 2:, 3]) if math.isnan(value) else got[i, 2:, 3] == value).all()
            rest = np.arange(dim) != 3
            assert (np.abs(got[i, 2:] - ref[i, 2:])[:, rest] <= tol[i, 2:][:, rest]).all()
        elif what == "v" or math.isnan(value):
            assert np.isnan(got[i, 2:]).all()
    assert np.array_equal(got[q[0]:], clean[q[0]:])


def test_attention_over_a_cache_past_32_bits(dv):
    """Pages whose element offsets pass 2^31 and byte offsets 2^32, bf16."""
    page, heads, dim = 128, 8, 128
    n_pages = 2 ** 31 // (page * heads * dim) + 200
    k = torch.empty((n_pages, heads, page, dim), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    st = Setup(dv, [1, 40], [500, 300], heads, dim, page, "bf16", seed=4)
    far = torch.arange(st.n_pages, dtype=torch.int64) + n_pages - st.n_pages
    k[-st.n_pages:] = st.cache.k
    v[-st.n_pages:] = st.cache.v
    small = st.cache
    st.cache = dv.KvCache(k, v)
    table = st.chunks.table
    table.copy_(torch.where(table >= 0, table + (n_pages - st.n_pages), table))
    q = st.queries(heads)
    got, status = dv.cache_attention(st.cache, st.chunks, q)
    rk, rv, status2 = dv.cache_read(st.cache, st.chunks, st.rows)
    st.cache = small
    table.copy_(st.table)
    want, _ = dv.cache_attention(small, st.chunks, q)
    wk, wv, _ = dv.cache_read(small, st.chunks, st.rows)
    torch.cuda.synchronize()
    assert int(status.item()) == dv.OK and int(status2.item()) == dv.OK and int(far[-1]) == n_pages - 1
    assert torch.equal(got, want) and torch.equal(rk, wk) and torch.equal(rv, wv)


def test_attention_one_pass_over_splits_is_repeatable(dv):
    """The same call twice gives the same bits, whatever was left in the workspace."""
    st = Setup(dv, [1, 3, 1], [5000, 2000, 17], 2, 128, 64, "bf16", seed=2)
    q = st.queries(8)
    a, _ = dv.cache_attention(st.cache, st.chunks, q)
    import ctypes
    nb = ctypes.c_size_t()
    dv.check(dv.lib.ds_vit_cache_attention_workspace_bytes(st.cache.ref, st.chunks.ref, 8, ctypes.byref(nb)), "size")
    ws = torch.full((nb.value,), 255, dtype=torch.uint8, device="cuda")
    b, _ = dv.cache_attention(st.cache, st.chunks, q, ws=ws)
    torch.cuda.synchronize()
    assert torch.equal(a, b)


def sampled64(st, q, scale, rows, window=0, sinks=0):
    """(reference, tolerance) [len(rows), heads, dim] of some packed rows, in 64
    bits on the GPU; the tolerance of attention64."""
    heads = q.shape[1]
    g = heads // st.kv_heads
    held = [torch.from_numpy(x).cuda() for x in st.held()]
    refs, tols = [], []
    for r in rows:
        s = max(i for i in range(len(st.q)) if st.off[i] <= r)
        p = st.kv[s] - st.q[s] + r - st.off[s]
        j = torch.arange(p + 1)
        if window:
            j = j[(j > p - window) | (j < sinks)]
        page, slot = st.table[s][j // st.page].long().cuda(), (j % st.page).cuda()
        k, v = (x[page, :, slot].repeat_interleave(g, 1) for x in held)          # [keys, heads, dim]
        x = q[r].double()
        z = torch.einsum("jhd,hd->hj", k, x) * scale
        w = torch.softmax(z, 1)
        ref = torch.einsum("hj,jhd->hd", w, v)
        big = torch.einsum("jhd,hd->hj", k.abs(), x.abs()).amax(1, keepdim=True) * scale
        refs.append(ref)
        tols.append(2.0 ** -8 * ref.abs() + torch.einsum("hj,jhd->hd", w, v.abs())
                    * (2.0 ** -8 + 2.0 ** -12 + 2 * (st.dim + 2) * 2.0 ** -24 * big))
    return torch.stack(refs).cpu().numpy(), torch.stack(tols).cpu().numpy()


LARGE = [
    # q, kv, heads, kv_heads, dim, page, kind, window, sinks
    ([900, 1300, 5], [9000, 1300, 4100], 8, 2, 128, 64, "bf16", 0, 0),          # many items a CTA, some of them split
    ([900, 1300, 5], [9000, 1300, 4100], 8, 2, 128, 64, "e4m3", 0, 0),
    ([2100], [2100], 12, 4, 64, 16, "bf16", 0, 0),                               # whole items
    ([1500, 700], [6000, 2000], 10, 2, 64, 128, "e4m3", 600, 3),
    ([400] * 20, [400 + 37 * i for i in range(20)], 6, 2, 128, 32, "bf16", 300, 20),
    ([3] * 150, [3 + 11 * i for i in range(150)], 21, 1, 64, 32, "e4m3", 0, 0),  # 63 rows an item, other key tiles to tile B
    ([3] * 150, [3 + 11 * i for i in range(150)], 21, 1, 128, 32, "bf16", 0, 0),
    ([30], [20011], 4, 1, 128, 64, "bf16", 0, 0),                                # few rows over many keys: split and shared
    ([30], [20011], 4, 1, 64, 16, "e4m3", 0, 0),
    ([30], [20011], 4, 1, 128, 16, "e4m3", 0, 0),
    ([1] * 60, [7000 - 111 * i for i in range(60)], 16, 4, 128, 64, "e4m3", 0, 0),
    ([1] * 60, [7000 - 111 * i for i in range(60)], 16, 4, 64, 32, "bf16", 2000, 4),
    ([1], [60007], 8, 1, 128, 128, "e4m3", 0, 0),                                # one item over every worker
    ([1], [60007], 16, 1, 64, 16, "bf16", 0, 0),
]


@pytest.mark.parametrize("q,kv,heads,kv_heads,dim,page,kind,window,sinks", LARGE)
def test_attention_of_larger_calls(dv, q, kv, heads, kv_heads, dim, page, kind, window, sinks):
    """Calls that give every worker several items or a part of one: sampled rows
    against 64 bits, and the same bits again over a workspace of other contents."""
    st = Setup(dv, q, kv, kv_heads, dim, page, kind, seed=sum(q) % 1000, fill=math.nan)
    x = st.queries(heads, wide=3)
    ws = torch.full((dv.cache_attention_workspace_bytes(st.cache, st.chunks, heads),), 255, dtype=torch.uint8,
                    device="cuda")
    got, status = dv.cache_attention(st.cache, st.chunks, x, window=window, sinks=sinks)
    again, _ = dv.cache_attention(st.cache, st.chunks, x, window=window, sinks=sinks, ws=ws)
    torch.cuda.synchronize()
    assert int(status.item()) == dv.OK
    assert torch.equal(got, again)
    rng = np.random.default_rng(5)
    rows = sorted({0, st.rows - 1, *rng.integers(0, st.rows, 40).tolist(),
                   *(st.off[s + 1] - 1 for s in range(0, len(q), 13))})
    ref, tol = sampled64(st, x, dim ** -0.5, rows, window, sinks)
    err = np.abs(f64(got)[rows] - ref)
    bad = ~(err <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size} outside, worst {np.nanmax(err / tol)} at {np.argwhere(bad)[:3].tolist()}"


COLD = [
    # q, kv, heads, kv_heads, page
    ([3] * 12, [6000 + 7 * i for i in range(12)], 32, 4, 64),        # 24 rows a K/V head
    ([1] * 24, [5000 - 90 * i for i in range(24)], 32, 4, 16),       # 8
    ([16], [20000], 64, 2, 32),                                      # 512, one sequence
    ([300, 41], [4000, 9000], 16, 2, 128),                           # whole tiles and a part of one
    ([8 + 9 * i % 76 for i in range(56)], [90 + 41 * i % 537 for i in range(56)], 64, 4, 32),   # one key tile and several, in turn
    ([3] * 200, [3 + 7 * i % 300 for i in range(200)], 42, 2, 16),   # 63 rows over one to three key tiles
]


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q,kv,heads,kv_heads,page", COLD)
def test_same_bits_from_cold_caches(dv, q, kv, heads, kv_heads, page, dim, kind):
    """Pages that come late (nothing of them in L2) and early: every wait holds
    whatever lands first, and the bits are the same."""
    st = Setup(dv, q, kv, kv_heads, dim, page, kind, seed=dim + len(q), fill=math.nan)
    x = st.queries(heads)
    flush = torch.empty(300 << 20, dtype=torch.uint8, device="cuda")
    first, status = dv.cache_attention(st.cache, st.chunks, x)
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(24):
        if i % 2 == 0:
            flush.fill_(i)
        got, _ = dv.cache_attention(st.cache, st.chunks, x, status=status)
        differ += (got != first).sum()
    torch.cuda.synchronize()
    assert int(status.item()) == dv.OK
    assert bool(torch.isfinite(first).all()) and int(differ.item()) == 0


@pytest.mark.parametrize("rows,heads", [(1, 8), (40, 8)])
def test_sequences_that_share_pages(dv, rows, heads):
    """Two sequences over the same pages (a common prompt) with the same queries
    give the same rows."""
    st = Setup(dv, [rows, rows], [300, 300], 2, 128, 16, "e4m3", seed=15)
    st.chunks.table[1] = st.chunks.table[0]
    x = st.queries(heads)
    x[rows:] = x[:rows]
    got, status = dv.cache_attention(st.cache, st.chunks, x)
    torch.cuda.synchronize()
    assert int(status.item()) == dv.OK and torch.equal(got[:rows], got[rows:])


@pytest.mark.parametrize("rows", [1, 60])
def test_two_streams_at_once(dv, rows):
    """Calls on two streams that overlap on the GPU, with the workspaces that the
    cache keeps for each."""
    st = Setup(dv, [rows] * 3, [4000, 2500, 900], 2, 128, 64, "bf16", seed=16)
    x = st.queries(8)
    want, _ = dv.cache_attention(st.cache, st.chunks, x)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.zeros_like(want) for _ in range(6)] for _ in streams]
    status = [torch.zeros(1, dtype=torch.int32, device="cuda") for _ in streams]
    torch.cuda.synchronize()
    for i in range(6):
        for s, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                dv.cache_attention(st.cache, st.chunks, x, out=outs[s][i], status=status[s])
    torch.cuda.synchronize()
    for s in range(2):
        assert int(status[s].item()) == dv.OK
        for o in outs[s]:
            assert torch.equal(o, want)


@pytest.mark.parametrize("rows", [1, 20, 140])
@pytest.mark.parametrize("q_exp,k_exp,v_exp", [(-60, 20, -70), (40, -60, 60), (0, 0, 100), (-100, 90, -100)])
def test_e4m3_far_exponents(dv, rows, q_exp, k_exp, v_exp):
    """Queries, keys and values many powers of two from one: the result scales with
    them.  Not bit for bit: the running reference (score plus exponent, fp32) rounds
    otherwise with other exponents, which scales the weights and their sum by one
    common factor 2^d, |d| <= 128 2^-24, and so moves the weights' own rounding.  Both
    results stay within attention64's tolerance of one and the same value, so
    they differ by at most twice that."""
    st = Setup(dv, [rows], [700], 1, 128, 16, "e4m3", seed=17)
    x = st.queries(4)
    scale = 128 ** -0.5
    want, _ = dv.cache_attention(st.cache, st.chunks, x, scale=scale)
    ke, ve = st.cache.k_exp.int() + k_exp, st.cache.v_exp.int() + v_exp
    assert int(ke.min()) >= 10 and int(ke.max()) <= 247 and int(ve.min()) >= 10 and int(ve.max()) <= 247
    far = dv.KvCache(st.cache.k, st.cache.v, ke.to(torch.uint8), ve.to(torch.uint8))
    got, status = dv.cache_attention(far, st.chunks, (x.float() * 2.0 ** q_exp).bfloat16(),
                                     scale=scale * 2.0 ** -(q_exp + k_exp))
    torch.cuda.synchronize()
    assert int(status.item()) == dv.OK
    picks = sorted({0, rows // 2, rows - 1})
    _, tol = sampled64(st, x, scale, picks)
    assert (np.abs(f64(got)[picks] * 2.0 ** -v_exp - f64(want)[picks]) <= 2 * tol).all()


# ------------------------------------------------------------------ entries refused on the device

def _calls(dv, st, heads=4):
    k = st.queries(st.kv_heads)
    yield lambda: dv.cache_write(st.cache, st.chunks, k, k)
    yield lambda: dv.cache_read(st.cache, st.chunks, st.rows)[2]
    q = st.queries(heads)
    yield lambda: dv.cache_attention(st.cache, st.chunks, q)[1]


@pytest.mark.parametrize("rows", [1, 60])
def test_entries_refused_on_the_device(dv, rows):
    """Bad offsets, lengths and pages set the status, and the other sequences are
    served as ever."""
    def make():
        return Setup(dv, [rows, rows, rows], [100, 90, 120], 2, 128, 16, "bf16", seed=11)

    def expect(st, code):
        for call in _calls(dv, st):
            status = call()
            torch.cuda.synchronize()
            assert int(status.item()) == code

    st = make()
    expect(st, dv.OK)
    for entry in (-1, st.n_pages, 2 ** 31 - 1, -2 ** 31):
        st = make()
        st.chunks.table[1, (90 - 1) // 16] = entry
        expect(st, dv.ERANGE)
    for value in (-1, 16 * st.table.shape[1] + 1, 2 ** 31 - 1, -2 ** 31):
        st = make()
        st.chunks.kv_len[1] = value
        expect(st, dv.ERANGE)
    for at, value in ((1, -5), (1, 2 ** 31 - 1), (3, 3 * rows + 1), (0, -1), (2, 0), (2, -2 ** 31)):
        st = make()
        st.chunks.row_off[at] = value
        expect(st, dv.EINVAL)
    st = make()
    q = st.queries(4)
    want, _ = dv.cache_attention(st.cache, st.chunks, q)
    st.chunks.table[1, 0] = -1
    got, status = dv.cache_attention(st.cache, st.chunks, q)
    torch.cuda.synchronize()
    assert int(status.item()) == dv.ERANGE
    assert torch.equal(got[:rows], want[:rows]) and torch.equal(got[2 * rows:], want[2 * rows:])


def test_more_rows_than_max_rows_refused(dv):
    st = Setup(dv, [4, 2], [40, 30], 2, 64, 16, "bf16", seed=12, max_rows=3)
    q = st.queries(4)
    got, status = dv.cache_attention(st.cache, st.chunks, q)
    torch.cuda.synchronize()
    assert int(status.item()) == dv.EINVAL
    ref, tol = attention64(st, q, 64 ** -0.5)
    assert (np.abs(f64(got)[4:] - ref[4:]) <= tol[4:]).all()


def test_no_rows_and_sequences_without_rows(dv):
    st = Setup(dv, [0, 0], [40, 0], 2, 64, 16, "bf16", seed=18)
    x = st.queries(4)
    assert x.shape[0] == 0
    dv.cache_write(st.cache, st.chunks, st.queries(2), st.queries(2))
    dv.cache_read(st.cache, st.chunks, 0)
    out, status = dv.cache_attention(st.cache, st.chunks, x)
    st = Setup(dv, [0, 0, 0], [40, 0, 7], 2, 64, 16, "bf16", seed=18, front=2, back=3)
    for heads in (4, 64):
        check_attention(dv, st, heads)
    torch.cuda.synchronize()
    assert out.shape == (0, 4, 64) and int(status.item()) == dv.OK


def test_binding_refuses_other_tensors(dv):
    """Types, shapes, strides and devices that the binding refuses before the call."""
    st = Setup(dv, [2, 3], [40, 30], 2, 64, 16, "bf16", seed=13)
    q, kv = st.queries(4), st.queries(2)
    cpu = dv.KvCache(st.cache.k.cpu(), st.cache.v.cpu())
    i32 = dict(dtype=torch.int32, device="cuda")
    bad = [lambda: dv.cache_write(st.cache, st.chunks, kv.float(), kv),
           lambda: dv.cache_write(st.cache, st.chunks, kv, kv[:4]),
           lambda: dv.cache_write(st.cache, st.chunks, kv[:, :1], kv),
           lambda: dv.cache_write(st.cache, st.chunks, kv.cpu(), kv),
           lambda: dv.cache_write(st.cache, st.chunks, kv.transpose(1, 2).contiguous().transpose(1, 2), kv),
           lambda: dv.cache_write(cpu, st.chunks, kv, kv),
           lambda: dv.cache_write(st.cache, st.chunks, kv, kv, status=torch.zeros(1, device="cuda")),
           lambda: dv.cache_write(st.cache, st.chunks, kv, kv, status=torch.zeros(1, dtype=torch.int32)),
           lambda: dv.cache_read(st.cache, st.chunks, 4, out=(kv, kv)),
           lambda: dv.cache_read(st.cache, st.chunks, 5, out=(kv, kv.half())),
           lambda: dv.cache_attention(st.cache, st.chunks, q[:, :3]),
           lambda: dv.cache_attention(st.cache, st.chunks, q[..., :32]),
           lambda: dv.cache_attention(st.cache, st.chunks, q.view(5, 256)),
           lambda: dv.cache_attention(st.cache, st.chunks, q, out=q[:4].clone()),
           lambda: dv.cache_attention(st.cache, st.chunks, q, scale=0.0),
           lambda: dv.cache_attention(st.cache, st.chunks, q, ws=torch.empty(16, dtype=torch.uint8, device="cuda")),
           lambda: dv.cache_attention(st.cache, st.chunks, q, ws=torch.empty(1 << 24, device="cuda")),
           lambda: dv.cache_attention(st.cache, dv.Chunks(torch.zeros(2, **i32).cpu(), torch.zeros(1, **i32).cpu(),
                                                          torch.zeros((1, 1), **i32).cpu(), 1), q)]
    for i, call in enumerate(bad):
        with pytest.raises(dv.DsVitError):
            call()
            pytest.fail(f"call {i} was not refused")


# ------------------------------------------------------------------ as a serving loop uses them

@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_prompt_with_an_image_in_chunks_then_tokens(dv, kind):
    """Two prompts with image spans: their rows are overlaid chunk by chunk, projected, written
    to the cache and attended; then single tokens follow.  Every attention equals the
    definition over what the cache holds, and the keys read back are those written."""
    width, heads, kv_heads, dim, page = 512, 12, 2, 64, 16
    n_out = (heads + 2 * kv_heads) * dim
    g = torch.Generator().manual_seed(21)
    w = (torch.randn((n_out, width), generator=g) / math.sqrt(width)).bfloat16().cuda()
    bias = (0.1 * torch.randn(n_out, generator=g)).bfloat16().cuda()
    embeds = torch.randn((12, width), generator=g).bfloat16().cuda()
    sentinel = torch.randn((3, width), generator=g).bfloat16().cuda()
    prompts = [torch.randn((70, width), generator=g).bfloat16().cuda() for _ in range(2)]
    spans = [[(20, 9, 6, 0)], [(41, 6, 9, 6)]]          # 3 x 2 and 2 x 3 merged tokens
    plan = [[(0, 33), (0, 20)], [(33, 60), (20, 70)], [(60, 70), (70, 70)], [(70, 71), (70, 71)], [(71, 72), (71, 72)]]
    total = 80
    st = Setup(dv, [1, 1], [total, total], kv_heads, dim, page, kind, seed=22)
    st.spoil(math.nan)
    ws = None
    written = [[], []]
    for step in plan:
        parts, lens = [], []
        for s, (a, b) in enumerate(step):
            if b <= 70:
                rows = prompts[s][a:b].clone()
                if b > a:
                    dv.overlay_chunk(rows, a, spans[s], embeds, sentinel)
            else:
                rows = torch.randn((b - a, width), generator=g).bfloat16().cuda()
            parts.append(rows)
            lens.append(b)
        x = torch.cat(parts)
        st.q, st.kv = [b - a for a, b in step], lens
        st.off = [0, st.q[0], sum(st.q)]
        st.rows = st.off[-1]
        st.chunks = dv.Chunks(torch.tensor(st.off, dtype=torch.int32).cuda(),
                              torch.tensor(lens, dtype=torch.int32).cuda(), st.table.cuda(), max(st.q))
        qkv, lst = dv.op_linear(x, w, bias)
        qkv = qkv.view(st.rows, heads + 2 * kv_heads, dim)
        q, k, v = qkv[:, :heads], qkv[:, heads:heads + kv_heads], qkv[:, heads + kv_heads:]
        status = dv.cache_write(st.cache, st.chunks, k, v)
        out, _ = dv.cache_attention(st.cache, st.chunks, q, ws=ws, status=status)
        torch.cuda.synchronize()
        assert int(status.item()) == dv.OK and int(lst.item()) == dv.OK
        ref, tol = attention64(st, q, dim ** -0.5)
        assert (np.abs(f64(out) - ref) <= tol).all()
        for s in range(2):
            written[s].append(f64(k)[st.off[s]:st.off[s + 1]])
    all_rows = dv.Chunks(torch.tensor([0, 72, 144], dtype=torch.int32).cuda(),
                         torch.tensor([72, 72], dtype=torch.int32).cuda(), st.table.cuda(), 72)
    rk, _, status = dv.cache_read(st.cache, all_rows, 144)
    torch.cuda.synchronize()
    assert int(status.item()) == dv.OK
    for s in range(2):
        want = np.concatenate([x for x in written[s] if len(x)])
        if kind == "e4m3":
            b, e = quantise(want)
            want = E4M3[b] * 2.0 ** (e[..., None].astype(float) - 127)
        assert np.array_equal(f64(rk)[72 * s:72 * s + 72], want)


@pytest.mark.parametrize("rows", [1, 50])
def test_captured_and_replayed_on_other_lengths(dv, rows):
    """Two graphs with a workspace each, replayed at the same time on two streams
    after their lengths, tables and queries changed."""
    sets = []
    for seed in (31, 32):
        st = Setup(dv, [rows, rows], [900, 300], 2, 128, 32, "e4m3" if seed == 31 else "bf16", seed=seed)
        q, k = st.queries(8), st.queries(2)
        out = torch.zeros((st.rows, 8, 128), dtype=torch.bfloat16, device="cuda")
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        sets.append((st, q, k, out, status))
    graphs, streams = [], []
    for st, q, k, out, status in sets:
        stream = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.graph(graph, stream=stream):
            dv.cache_write(st.cache, st.chunks, k, k, status=status)
            dv.cache_attention(st.cache, st.chunks, q, out=out, status=status)
        graphs.append(graph)
        streams.append(stream)
    for lens in ([900, 300], [rows, 896], [513, rows + 1]):
        for st, q, k, out, status in sets:
            st.kv = lens
            free = torch.randperm(st.n_pages, generator=st.g).int()
            used = [-(-x // 32) for x in lens]
            st.table.fill_(-1)
            for s in range(2):
                st.table[s, :used[s]] = free[sum(used[:s]):sum(used[:s + 1])]
            st.chunks.table.copy_(st.table)
            st.chunks.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
            q.copy_(torch.randn(q.shape, generator=st.g))
            k.copy_(torch.randn(k.shape, generator=st.g))
        torch.cuda.synchronize()
        for _ in range(3):
            for graph, stream in zip(graphs, streams):
                with torch.cuda.stream(stream):
                    graph.replay()
        torch.cuda.synchronize()
        for st, q, k, out, status in sets:
            assert int(status.item()) == dv.OK
            ref, tol = attention64(st, q, 128 ** -0.5)
            assert (np.abs(f64(out) - ref) <= tol).all()


# ------------------------------------------------------------------ rows of zeros

def put_tokens(st, s, j, k=None, v=None):
    """Keys and values (float64 [tokens, kv_heads, dim]) of tokens j of sequence s, as a write leaves them."""
    at = torch.from_numpy(st.table[s].numpy()[j // st.page]).long().cuda(), torch.from_numpy(j % st.page).cuda()
    for x, t, e in ((k, st.cache.k, st.cache.k_exp), (v, st.cache.v, st.cache.v_exp)):
        if x is None:
            continue
        x = torch.from_numpy(np.ascontiguousarray(x)).bfloat16()
        if e is None:
            t[at[0], :, at[1]] = x.cuda()
        else:
            b, ex = quantise(x.double().numpy())
            t[at[0], :, at[1]] = torch.from_numpy(b).cuda()
            e[at[0], :, at[1]] = torch.from_numpy(ex).cuda()


ZERO_LAYOUTS = [
    # q, kv, heads, kv_heads, page
    ([1], [1100], 8, 1, 64),                  # one token, one worker's blocks and a few
    ([1, 1], [60007, 300], 8, 1, 128),        # a long one over every worker
    ([4, 1], [900, 260], 6, 2, 16),           # a few rows
    ([40], [900], 4, 2, 32),                  # chunks
    ([300, 20], [1500, 700], 4, 1, 64),
    ([30], [20011], 4, 1, 64),                # a chunk's items split between workers
]


@pytest.mark.parametrize("form", ["first", "middle", "last", "none seen", "all", "all rising", "rising"])
@pytest.mark.parametrize("kind,dim", [("e4m3", 128), ("e4m3", 64), ("bf16", 128)])
@pytest.mark.parametrize("q,kv,heads,kv_heads,page", ZERO_LAYOUTS)
def test_attention_over_zero_rows(dv, q, kv, heads, kv_heads, page, kind, dim, form):
    """Tokens whose values (and keys) are zeros, as padding and placeholders leave them: they
    keep their weight in the sum, wherever they lie and however the scores run."""
    st = Setup(dv, q, kv, kv_heads, dim, page, kind, seed=len(form) + dim)
    x = st.queries(heads)
    scale = dim ** -0.5
    g = np.random.default_rng(7)
    for s, n in enumerate(kv):
        j = np.arange(n)
        if form.endswith("rising"):           # positive scores that rise by some 40 (58 in powers of two)
            base = np.abs(g.standard_normal((1, kv_heads, dim)))
            put_tokens(st, s, j, k=base * ((j + 1) / n)[:, None, None])
        some = {"first": j < max(n // 3, 128), "middle": (j >= n // 4) & (j < n // 4 + max(n // 2, 1)),
                "last": j >= n - max(n // 3, 130), "none seen": j < n - q[s], "all": j >= 0, "all rising": j >= 0,
                "rising": j < n - n // 5}[form]
        z = np.zeros((int(some.sum()), kv_heads, dim))
        put_tokens(st, s, j[some], k=z if form in ("first", "middle", "last") else None, v=z)
    if form.endswith("rising"):
        x, scale = x.abs(), 40 / (dim * 2 / math.pi)
    out = torch.full((st.rows, heads, dim), 7.0, dtype=torch.bfloat16, device="cuda")
    got, status = dv.cache_attention(st.cache, st.chunks, x, scale=scale, out=out)
    torch.cuda.synchronize()
    assert int(status.item()) == dv.OK
    rows = sorted({0, st.rows - 1, st.rows // 2, *(st.off[s] for s in range(len(q)))})
    ref, tol = sampled64(st, x, scale, rows)
    bad = ~(np.abs(f64(got)[rows] - ref) <= tol)
    assert not bad.any(), f"{bad.sum()} of {bad.size} outside, {f64(got)[rows][bad][:3]} for {ref[bad][:3]}"
    if form.startswith("all"):
        assert bool((got == 0).all())


# ------------------------------------------------------------------ rows far apart

def far64(st, q, scale, rows, window=0, sinks=0):
    """(reference, tolerance) [len(rows), heads, dim] in 64 bits where keys or values lie
    far apart, e4m3.  As attention64's tolerance, but a score's error goes by its own key:
    each weight w_j is off by (dim + 2) 2^-24 sum_d |q_d k_jd| of itself, and so is their
    sum, weighed by w_j.  To this comes what fp16 operands lose under 2^-14: with the
    reference at most 2^8 above the row's largest contribution c = max w_j 2^e_j (and that one
    taken to 2^6 or more), up to 2^-25 / 2^-2 c of every operand, whose products are with the
    elements v_j 2^-e_j."""
    heads = q.shape[1]
    g = heads // st.kv_heads
    held = [torch.from_numpy(x).cuda() for x in st.held()]
    e = st.cache.v_exp.double() - 127
    refs, tols = [], []
    for r in rows:
        s = max(i for i in range(len(st.q)) if st.off[i] <= r)
        p = st.kv[s] - st.q[s] + r - st.off[s]
        j = torch.arange(p + 1)
        if window:
            j = j[(j > p - window) | (j < sinks)]
        page, slot = st.table[s][j // st.page].long().cuda(), (j % st.page).cuda()
        k, v = (x[page, :, slot].repeat_interleave(g, 1) for x in held)          # [keys, heads, dim]
        ej = torch.exp2(e[page, :, slot].repeat_interleave(g, 1))                # [keys, heads]
        x = q[r].double()
        w = torch.softmax(torch.einsum("jhd,hd->jh", k, x) * scale, 0)
        eps = (st.dim + 2) * 2.0 ** -24 * torch.einsum("jhd,hd->jh", k.abs(), x.abs()) * scale
        # a factor exp(eps) - 1 where eps is not small; a weight of at most 2^-200 is nothing whatever its error
        eps = torch.where(w > 2.0 ** -200, torch.expm1(eps), torch.zeros_like(eps))
        ref = torch.einsum("jh,jhd->hd", w, v)
        size = torch.einsum("jh,jhd->hd", w, v.abs())
        most = (w * ej).amax(0)[:, None]
        refs.append(ref)
        tols.append(2.0 ** -8 * ref.abs() + size * (2.0 ** -8 + 2.0 ** -12 + torch.einsum("jh,jh->h", w, eps)[:, None])
                    + torch.einsum("jh,jhd->hd", w * eps, v.abs())
                    + 2.0 ** -23 * most * torch.einsum("jh,jhd->hd", 1 / ej, v.abs()))
    return torch.stack(refs).cpu().numpy(), torch.stack(tols).cpu().numpy()


@pytest.mark.parametrize("far", [10, 20, 40])
@pytest.mark.parametrize("form", ["hidden k", "hidden v", "hidden both", "seen k", "seen v", "zeros"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q,kv,heads,kv_heads,page,window,sinks", [
    ([4, 1], [900, 260], 6, 2, 16, 0, 0),
    ([40], [900], 4, 2, 32, 0, 0),
    ([300], [900], 2, 1, 64, 0, 0),
    ([300, 20], [1500, 700], 4, 1, 16, 200, 3),
    ([30], [20011], 4, 1, 64, 0, 0),
])
def test_attention_over_rows_far_apart(dv, q, kv, heads, kv_heads, page, window, sinks, dim, form, far):
    """A finite key or value 2^far times the others', hidden from some rows of its tile or seen
    with next to no weight, takes nothing from the keys beside it; nor does a row of zeros
    with the largest score beside such a value."""
    st = Setup(dv, q, kv, kv_heads, dim, page, "e4m3", seed=far + dim)
    x = st.queries(heads).abs()               # so that a sign decides a score
    scale = dim ** -0.5
    g = np.random.default_rng(far)
    one = lambda f: f * np.abs(g.standard_normal((1, kv_heads, dim)))   # noqa: E731
    for s, n in enumerate(kv):
        c = q[s]
        if form.startswith("hidden"):
            # a later token of the chunk; every row before it, and (window) rows far behind it, do not see it
            for at in (n - c + c // 2, n - c):
                put_tokens(st, s, np.array([at]), k=one(2.0 ** far) if form != "hidden v" else None,
                           v=one(2.0 ** far) if form != "hidden k" else None)
        else:
            for at in (5, n - c - 7, n - c // 2):
                if at >= n - 1:
                    continue
                put_tokens(st, s, np.array([at]), k=one(-2.0 ** far if form == "seen k" else -12.0),
                           v=one(2.0 ** far) if form != "seen k" else None)
                if form == "zeros":
                    put_tokens(st, s, np.array([at + 1]), k=one(3.0), v=one(0.0))
    got, status = dv.cache_attention(st.cache, st.chunks, x, scale=scale, window=window, sinks=sinks)
    torch.cuda.synchronize()
    assert int(status.item()) == dv.OK
    rows = sorted({0, st.rows - 1, *(st.off[s] + min(i, q[s] - 1) for s in range(len(q))
                                     for i in (0, 1, q[s] // 4, q[s] // 2 - 1, q[s] // 2, 200, q[s] - 1) if i >= 0)})
    ref, tol = far64(st, x, scale, rows, window, sinks)
    err = np.abs(f64(got)[rows] - ref)
    bad = ~(err <= tol)
    assert not bad.any(), (f"{bad.sum()} of {bad.size} outside, worst {np.nanmax(err / tol)}, "
                           f"rows {sorted({rows[i] for i in np.argwhere(bad)[:, 0]})}")


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 5)])
def test_same_bits_over_many_calls(dv, dim, kind, window, sinks):
    """Ragged chunks of few key tiles: a warp that is done with its item's last tile while others
    are two products behind must not take an earlier product's completion for its last one's."""
    q, kv = [8 + 9 * i % 76 for i in range(56)], [90 + 41 * i % 537 for i in range(56)]
    st = Setup(dv, q, kv, 4, dim, 32, kind, seed=dim + len(q), fill=math.nan)
    x = st.queries(64)
    flush = torch.empty(300 << 20, dtype=torch.uint8, device="cuda")
    first, status = dv.cache_attention(st.cache, st.chunks, x, window=window, sinks=sinks)
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(600):
        if i % 2 == 0:
            flush.fill_(i % 251)
        got, _ = dv.cache_attention(st.cache, st.chunks, x, window=window, sinks=sinks, status=status)
        differ += (got != first).sum()
    torch.cuda.synchronize()
    assert int(status.item()) == dv.OK
    assert bool(torch.isfinite(first).all()) and int(differ.item()) == 0


@pytest.mark.parametrize("first", [1, 3])
@pytest.mark.parametrize("q,kv,dim,window,sinks", [([4], [200], 128, 0, 0), ([4], [200], 64, 20, 3),
                                                   ([70], [300], 128, 0, 0), ([70], [300], 64, 30, 5),
                                                   ([70, 70], [300, 70], 128, 0, 0)])
def test_first_scores_of_minus_infinity(dv, q, kv, dim, window, sinks, first):
    """Keys with an infinity against the query weigh nothing, in rows too that are computed
    again because a value hidden from them is not finite."""
    st = Setup(dv, q, kv, 2, dim, 16, "bf16", seed=9)
    x = st.queries(4)
    x[..., 3] = x[..., 3].abs() + 0.5
    for j in range(first):
        _plant(st, 0, j, 1, -math.inf, "k")
    bad = kv[0] - q[0] + q[0] // 2
    _plant(st, 0, bad, 1, math.nan, "v")
    got, status = dv.cache_attention(st.cache, st.chunks, x, window=window, sinks=sinks)
    torch.cuda.synchronize()
    assert int(status.item()) == dv.OK
    got = f64(got)
    # the definition without those keys, with attention64's tolerance; the infinity's element plays no part in it
    k, v = (y[:, 1] for y in (st.tokens(h, 0) for h in st.held()))
    for i in (0, q[0] // 2 - 1):
        p = kv[0] - q[0] + i
        j = np.arange(first, p + 1)
        if window:
            j = j[(j > p - window) | (j < sinks)]
        for h in (2, 3):
            qq = f64(x[i, h])
            z = k[j] @ qq * dim ** -0.5
            w = np.exp(z - z.max())
            w /= w.sum()
            big = (np.abs(k[j]) @ np.abs(qq)).max() * dim ** -0.5
            ref = w @ v[j]
            tol = 2.0 ** -8 * np.abs(ref) + (w @ np.abs(v[j])) * (2.0 ** -8 + 2.0 ** -12 + 2 * (dim + 2) * 2.0 ** -24 * big)
            assert (np.abs(got[i, h] - ref) <= tol).all()
    sees = [i for i in range(q[0] // 2, q[0]) if not window or bad > kv[0] - q[0] + i - window]
    assert np.isnan(got[sees, 2:, 3]).all()


@pytest.mark.parametrize("rows", [1, 40])
def test_two_threads_on_one_stream(dv, rows):
    """Threads whose calls, split between workers, come between one another's launches on the
    default stream."""
    import threading
    sets = []
    for seed, n in ((41, 9000), (42, 7000)):
        st = Setup(dv, [rows, rows + 1], [n, 300 + seed], 2, 128, 64, "bf16", seed=seed)
        x = st.queries(8)
        sets.append((st, x, dv.cache_attention(st.cache, st.chunks, x)[0]))
    torch.cuda.synchronize()
    start, wrong = threading.Barrier(2, timeout=60), [None, None]

    def thread(i):
        st, x, want = sets[i]
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        differ = torch.zeros((), dtype=torch.int64, device="cuda")
        start.wait()
        for _ in range(300):
            differ += (dv.cache_attention(st.cache, st.chunks, x, status=status)[0] != want).sum()
        wrong[i] = int(differ.item()), int(status.item())

    threads = [threading.Thread(target=thread, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert wrong == [(0, dv.OK)] * 2


@pytest.mark.parametrize("n,c,kv,heads,dim,kind", [
    (152, 2, 400000, 16, 64, "bf16"), (152, 2, 200000, 16, 128, "e4m3"),      # many rows: an item a CTA and more
    (1024, 2, 100000, 4, 128, "bf16"), (1024, 2, 100000, 8, 64, "e4m3"),      # few rows: several items a worker
    (2, 40, 150000, 4, 128, "bf16"), (1, 3, 300000, 4, 64, "e4m3"),           # items split between workers
])
def test_hidden_value_behind_a_long_cache(dv, n, c, kv, heads, dim, kind):
    """Rows to be computed again over long caches (shared by the sequences): it takes its time, and
    no wait runs into its limit meanwhile.  The newest token's value, seen by the last
    row alone, is not finite."""
    st = Setup(dv, [c], [kv], 1, dim, 128, kind, seed=19)
    rows = torch.randn((n * c, heads, dim), generator=st.g).bfloat16().cuda()
    off = torch.arange(0, n * c + 1, c, dtype=torch.int32, device="cuda")
    chunks = dv.Chunks(off, torch.full((n,), kv, dtype=torch.int32, device="cuda"),
                       st.table.cuda().expand(n, -1).contiguous(), c)
    clean, _ = dv.cache_attention(st.cache, chunks, rows)
    _plant(st, 0, kv - 1, 0, math.nan, "v")
    got, status = dv.cache_attention(st.cache, chunks, rows)
    torch.cuda.synchronize()
    assert int(status.item()) == dv.OK
    assert bool(torch.isnan(got[c - 1::c, :, 3]).all())
    hidden = torch.ones(n * c, dtype=torch.bool, device="cuda")
    hidden[c - 1::c] = False
    a, b = got[hidden].float(), clean[hidden].float()
    # Both within attention64's tolerance of one value, so at most twice that apart; of it, taken from
    # what is at hand: 2^-8 |o|, and A (2^-8 + 2^-12 + 2 (dim + 2) 2^-24 big) with the weighed mean size A of the
    # values and the largest sum |q_d k_d| scale, `big`, each bounded over all rows.
    assert bool(torch.isfinite(a).all())
    held = [torch.from_numpy(x).cuda() for x in st.held()]
    k, v = (st.tokens(x.cpu().numpy(), 0)[:kv - 1, 0] for x in held)
    picks = [0, int(hidden.nonzero()[-1])]
    for r in picks:
        s, i = divmod(r, c)
        p = kv - c + i
        kk, vv = torch.from_numpy(k[:p + 1]).cuda(), torch.from_numpy(v[:p + 1]).cuda()
        q = rows[r].double()
        w = torch.softmax(q @ kk.T * dim ** -0.5, 1)
        ref, size = w @ vv, w @ vv.abs()
        big = (q.abs() @ kk.abs().T).amax(1, keepdim=True) * dim ** -0.5
        tol = 2.0 ** -8 * ref.abs() + size * (2.0 ** -8 + 2.0 ** -12 + 2 * (dim + 2) * 2.0 ** -24 * big)
        assert bool(((got[r].double() - ref).abs() <= tol).all())
    # every row against the same of the clean call: rows of one position share keys, sizes are alike to a factor of two
    top = 2 * float(size.max())
    lim = 2 * (2.0 ** -8 * b.abs() + top * (2.0 ** -8 + 2.0 ** -12 + 2 * (dim + 2) * 2.0 ** -24 * 2 * float(big.max())))
    assert bool(((a - b).abs() <= lim).all())


@pytest.mark.parametrize("q,kv,kind", [([4, 1], [200, 90], "bf16"), ([70, 3], [300, 70], "bf16"), ([70, 3], [300, 70], "e4m3"),
                                       ([300], [2000], "bf16")])
def test_values_seen_and_hidden_that_are_not_finite(dv, q, kv, kind):
    """An infinity or NaN among the first tokens, seen by every row, stays in its elements; with
    another one hidden from the earlier rows, those have the first one's alone."""
    st = Setup(dv, q, kv, 2, 128, 16, kind, seed=23)
    x = st.queries(4)
    page, slot = int(st.table[0, 0]), 5
    if kind == "bf16":
        st.cache.v[page, 1, slot, 7] = math.inf
    seen, status = dv.cache_attention(st.cache, st.chunks, x)
    bad = kv[0] - q[0] // 2
    _plant(st, 0, bad, 1, math.nan, "v")
    both, _ = dv.cache_attention(st.cache, st.chunks, x, status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == dv.OK
    ref, tol = sampled64(st, x, 128 ** -0.5, rows := [0, q[0] // 4, bad - kv[0] + q[0] - 1])
    for i, r in enumerate(rows):
        for y in (seen, both):
            y = f64(y[r])
            if kind == "bf16":
                assert (y[2:, 7] == math.inf).all()
            rest = np.arange(128) != 7
            assert np.isfinite(y[:, rest]).all() and (np.abs(y - ref[i])[:, rest] <= tol[i][:, rest]).all()
    late = f64(both[bad - kv[0] + q[0]:q[0]])
    assert np.isnan(late[:, 2:, 3]).all() and np.isfinite(late[:, :2]).all()


def test_front_padding_beside_hidden_values(dv):
    """Rows in front of position 0 stay zeros beside tokens that are not finite."""
    for kind in ("bf16", "e4m3"):
        for heads in (4, 64):
            st = Setup(dv, [9, 40], [4, 30], 2, 64, 16, kind, seed=24)
            _plant(st, 0, 3, 1, math.nan, "v")
            _plant(st, 1, 20, 0, math.nan, "v")
            got, status = dv.cache_attention(st.cache, st.chunks, st.queries(heads))
            torch.cuda.synchronize()
            assert int(status.item()) == dv.OK
            got = f64(got)
            assert (got[:5] == 0).all() and (got[9:19] == 0).all() and np.isfinite(got[5:8]).all()


@pytest.mark.parametrize("bad", [dict(window=2 ** 32 + 5), dict(window=2 ** 31), dict(sinks=2 ** 32), dict(window=-1)])
def test_windows_past_32_bits_refused(dv, bad):
    st = Setup(dv, [2], [40], 2, 64, 16, "bf16", seed=13)
    with pytest.raises(dv.DsVitError):
        dv.cache_attention(st.cache, st.chunks, st.queries(4), **bad)

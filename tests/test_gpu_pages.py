"""Pages of many sequences on the GPU: resizing, releasing, forking and compacting
against a plain model of lists and counts, entry by entry, and the copies that go with them."""
import random

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


def up(x, page):
    return -(-x // page)


class Model:
    """The definition, one list entry after the other."""

    def __init__(self, n_pages, page, slots, cols):
        self.refs = np.zeros(n_pages, dtype=np.int64)
        self.table = np.full((slots, cols), -1, dtype=np.int64)
        self.len = np.zeros(slots, dtype=np.int64)
        self.page, self.n_pages = page, n_pages
        self.copies = []

    def free(self):
        return [int(p) for p in np.flatnonzero(self.refs == 0)]

    def drop(self, s, c):
        p = self.table[s, c]
        if p >= 0:
            self.refs[p] -= 1
        self.table[s, c] = -1

    def resize(self, slots, lengths, cap):
        grows = []
        for s, x in zip(slots, lengths):
            for c in range(up(x, self.page), up(self.len[s], self.page)):
                self.drop(s, c)
            if x > self.len[s]:
                grows.append((s, x))
            else:
                self.len[s] = x
        free, take, copies = self.free(), [], set()
        for s, x in grows:
            have = up(self.len[s], self.page)
            if self.len[s] % self.page and self.refs[self.table[s, have - 1]] > 1:
                take.append((s, have - 1))
                copies.add((s, have - 1))
            take += [(s, c) for c in range(have, up(x, self.page))]
        self.copies = []
        if len(take) > len(free) or len(copies) > cap:
            return False
        shared = [self.table[s, c] for s, c in copies]
        for (s, c), p in zip(take, free):
            if (s, c) in copies:
                self.copies.append((int(self.table[s, c]), p))
            self.table[s, c] = p
            self.refs[p] = 1
        for p in shared:
            self.refs[p] -= 1
        for s, x in grows:
            self.len[s] = x
        return True

    def release(self, slots, begin, end):
        for s, b, e in zip(slots, begin, end):
            for c in range(up(b, self.page), max(up(b, self.page), min(e, self.len[s]) // self.page)):
                self.drop(s, c)

    def fork(self, src, dst, cap):
        free = self.free()
        part = [s for s in src if self.len[s] % self.page and self.table[s, self.len[s] // self.page] >= 0]
        self.copies = []
        if len(part) > min(len(free), cap):
            return False
        for s, d in zip(src, dst):
            full = self.len[s] // self.page
            self.table[d, :full] = np.maximum(self.table[s, :full], -1)
            for p in self.table[d, :full]:
                if p >= 0:
                    self.refs[p] += 1
            if self.len[s] % self.page:
                p = self.table[s, full]
                self.table[d, full] = -1
                if p >= 0:
                    to = free.pop(0)
                    self.table[d, full] = to
                    self.refs[to] = 1
                    self.copies.append((int(p), to))
            self.len[d] = self.len[s]
        return True

    def compact(self, cap):
        used = int((self.refs > 0).sum())
        holes = np.flatnonzero(self.refs[:used] == 0)
        movers = used + np.flatnonzero(self.refs[used:] > 0)
        self.copies = [(int(a), int(b)) for a, b in zip(movers, holes)][:cap]
        now = np.arange(self.n_pages)
        for a, b in self.copies:
            self.refs[b], self.refs[a] = self.refs[a], 0
            now[a] = b
        for s in range(len(self.len)):
            t = self.table[s, :up(self.len[s], self.page)]
            t[:] = np.where(t >= 0, now[t], t)


class Both:
    def __init__(self, dv, n_pages, page, slots, cols, cap=None):
        self.dv, self.cap = dv, n_pages if cap is None else cap
        self.m = Model(n_pages, page, slots, cols)
        self.pool = dv.PagePool.empty(n_pages, page)
        self.tables = dv.PageTables.empty(slots, cols)
        self.copies = dv.PageCopies(self.cap)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def check(self, want=0, copies=True):
        torch.cuda.synchronize()
        assert int(self.status.item()) == want
        self.status.zero_()
        m = self.m
        assert np.array_equal(self.pool.refs.cpu().numpy(), m.refs)
        assert np.array_equal(self.tables.kv_len.cpu().numpy(), m.len)
        assert np.array_equal(self.tables.table.cpu().numpy(), m.table)
        if copies:
            n = int(self.copies.count.item())
            got = list(zip(self.copies.src[:n].tolist(), self.copies.dst[:n].tolist()))
            assert got == m.copies
        # the counts are those of the tables
        cols = np.arange(m.table.shape[1])[None] < up(m.len, m.page)[:, None]
        named = m.table[cols & (m.table >= 0)]
        assert np.array_equal(np.bincount(named, minlength=m.n_pages), m.refs)

    def i32(self, x):
        return torch.tensor(list(x), dtype=torch.int32, device="cuda")

    def resize(self, slots, lengths):
        self.dv.pages_resize(self.pool, self.tables, self.i32(slots), self.i32(lengths), self.copies, self.status)
        self.check(self.dv.OK if self.m.resize(slots, lengths, self.cap) else self.dv.ECAP)

    def release(self, slots, begin, end):
        self.dv.pages_release(self.pool, self.tables, self.i32(slots), self.i32(begin), self.i32(end), self.status)
        self.m.release(slots, begin, end)
        self.check(copies=False)

    def fork(self, src, dst):
        self.dv.pages_fork(self.pool, self.tables, self.i32(src), self.i32(dst), self.copies, self.status)
        self.check(self.dv.OK if self.m.fork(src, dst, self.cap) else self.dv.ECAP)

    def compact(self):
        self.dv.pages_compact(self.pool, self.tables, self.copies, self.status)
        self.m.compact(self.cap)
        self.check()


@pytest.mark.parametrize("n_pages", [1, 2, 3, 4, 5, 31, 37, 1000])
def test_small_pools(dv, n_pages):
    b = Both(dv, n_pages, 16, 4, n_pages)
    b.resize([2], [1])
    b.resize([2], [16 * n_pages])
    b.resize([2, 1], [17 if n_pages > 1 else 16, 0])
    b.resize([0, 2], [5, 0])
    b.resize([1], [16 * n_pages])          # one page is taken: not enough
    b.compact()
    b.resize([0, 1], [0, 16 * n_pages])    # what this call gives back can be taken by it


def test_beams(dv):
    b = Both(dv, 300, 16, 40, 30)
    b.resize([0, 1, 2, 3], [100, 160, 1, 0])
    src = [0, 0, 0, 1, 1, 2, 3]
    kids = list(range(10, 17))
    b.fork(src, kids)
    b.resize(kids[:6], [x + 1 for x in (100, 100, 100, 160, 160, 1)])
    b.resize(kids, [0] * 7)
    b.fork([1, 1, 1, 1, 2, 2, 0], kids)
    b.resize([0, 1, 2], [0, 0, 0])         # the children keep the pages
    b.compact()


def test_growing_in_a_shared_page_copies_it(dv):
    b = Both(dv, 50, 32, 6, 8)
    b.resize([0], [128])
    b.fork([0, 0], [1, 2])                 # nothing to copy: four full pages
    b.resize([1, 2], [70, 100])            # back to the middle of shared pages
    b.resize([1, 2], [71, 101])            # one copy each
    assert len(b.m.copies) == 2
    b.resize([0], [70])
    b.resize([0], [129])
    b.fork([0], [3])
    b.resize([0, 3], [66, 67])
    b.resize([0, 3], [68, 68])             # pages shared by these two alone
    b.resize([0, 1, 2, 3], [0, 0, 0, 0])
    assert not b.m.refs.any()


def test_copies_that_do_not_fit(dv):
    b = Both(dv, 50, 16, 8, 8, cap=1)
    b.resize([0, 1], [20, 21])
    b.fork([0, 1], [2, 3])
    assert b.m.len[2] == 0
    b.fork([0], [2])
    b.resize([0], [64])
    b.fork([0, 0], [3, 4])
    b.resize([3, 4], [50, 50])
    b.resize([3, 4], [51, 51])             # two copies, room for one
    b.resize([3], [51])


def test_releasing_behind_a_window(dv):
    b = Both(dv, 200, 16, 4, 60)
    b.resize([0, 1, 3], [900, 40, 7])
    b.release([0, 1, 3], [4, 0, 0], [500, 40, 7])        # a first page that stays; last pages not full stay
    b.release([0, 0, 0], [16, 100, 0], [600, 640, 17])   # overlapping, and what is gone already
    b.fork([0], [2])                                     # entries without a page are passed on
    b.release([2], [0], [900])
    b.compact()
    b.resize([0, 2], [0, 0])


@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_many_pages_of_unequal_sequences(dv, page):
    r = random.Random(page)
    n = 300
    lens = [int(3000 ** r.random()) for _ in range(n)]
    total = sum(up(x, page) for x in lens)
    b = Both(dv, total + 400, page, n + 200, up(3000, page) + 1)
    b.resize(list(range(n)), lens)
    gone = r.sample(range(n), 150)
    b.resize(gone, [r.choice([0, 0, x // 2]) for x in (lens[s] for s in gone)])
    kids = list(range(n, n + 200))
    b.fork([r.randrange(n) for _ in kids], kids)
    b.compact()
    b.compact()
    assert b.m.copies == []


def test_a_long_random_life(dv):
    r = random.Random(5)
    b = Both(dv, 400, 16, 60, 40, cap=37)
    for step in range(150):
        live = [s for s in range(60) if b.m.len[s]]
        idle = [s for s in range(60) if not b.m.len[s]]
        what = r.choice(["resize", "resize", "fork", "release", "compact"])
        if what == "resize":
            slots = r.sample(range(60), r.randint(1, 20))
            to = [r.choice([0, int(b.m.len[s]) + 1, min(640, int(b.m.len[s]) + r.randint(0, 60)), r.randint(0, 300)])
                  for s in slots]
            # a sequence whose last page was given away may not grow within it
            ok = [(s, min(x, 640)) for s, x in zip(slots, to) if x <= b.m.len[s] or b.m.len[s] % 16 == 0
                  or b.m.table[s, b.m.len[s] // 16] >= 0]
            if ok:
                b.resize(*zip(*ok))
        elif what == "fork" and live and idle:
            dst = r.sample(idle, r.randint(1, min(8, len(idle))))
            b.fork([r.choice(live) for _ in dst], dst)
        elif what == "release" and live:
            slots = [r.choice(live) for _ in range(r.randint(1, 6))]
            begin = [r.randint(0, 100) for _ in slots]
            b.release(slots, begin, [x + r.randint(0, 200) for x in begin])
        elif what == "compact":
            b.compact()


def test_a_large_pool(dv):
    """Stripes of several rounds, and lists as long as they may be."""
    n_pages, n = 1_000_003, 1024
    b = Both(dv, n_pages, 16, 3000, 1000, cap=100000)
    r = random.Random(9)
    b.resize(list(range(n)), [r.randint(1, 12000) for _ in range(n)])
    b.resize(r.sample(range(n), 500), [0] * 500)
    live = [s for s in range(n) if b.m.len[s]]
    b.fork([r.choice(live) for _ in range(n)], list(range(1500, 1500 + n)))
    b.compact()


def test_entries_left_out(dv):
    """Bad entries of a list are reported and left out; the others are served."""
    def fresh():
        b = Both(dv, 60, 16, 8, 5)
        b.resize([0, 1, 2], [33, 48, 5])
        return b

    b = fresh()                                       # a slot twice: both left out
    dv.pages_resize(b.pool, b.tables, b.i32([0, 3, 0]), b.i32([0, 7, 80]), b.copies, b.status)
    b.m.resize([3], [7], 60)
    b.check(dv.EINVAL)
    for slot, length in ((8, 3), (-1, 3), (4, 81), (4, -1), (2 ** 31 - 1, 1)):
        b = fresh()
        dv.pages_resize(b.pool, b.tables, b.i32([slot, 5]), b.i32([length, 17]), b.copies, b.status)
        b.m.resize([5], [17], 60)
        b.check(dv.ERANGE)
    b = fresh()                                       # the last page was given away
    b.tables.table[0, 2] = -1
    dv.pages_resize(b.pool, b.tables, b.i32([0, 5]), b.i32([34, 17]), b.copies, b.status)
    torch.cuda.synchronize()
    assert int(b.status.item()) == dv.ERANGE and b.tables.kv_len.tolist()[:6] == [33, 48, 5, 0, 0, 17]
    b = fresh()                                       # its full pages may have been
    b.tables.table[0, 0] = -1
    b.m.table[0, 0] = -1
    b.m.refs[0] = 0
    b.pool.refs[0] = 0
    b.resize([0], [34])
    for src, dst, why in (([0, 1], [4, 4], dv.EINVAL), ([0, 4], [4, 5], dv.EINVAL), ([0, 1], [1, 6], dv.EINVAL),
                          ([0, 8], [6, 7], dv.ERANGE), ([0, 1], [6, 9], dv.ERANGE), ([-1, 0], [6, 7], dv.ERANGE)):
        b = fresh()
        dv.pages_fork(b.pool, b.tables, b.i32(src), b.i32(dst), b.copies, b.status)
        keep = [(s, d) for s, d in zip(src, dst)
                if 0 <= s < 8 and 0 <= d < 8 and dst.count(d) == 1 and s not in dst and not b.m.len[d]]
        if keep:
            b.m.fork(*zip(*keep), 60)
        else:
            b.m.copies = []
        b.check(why)
    for begin, end, why in ((-1, 5, dv.ERANGE), (17, 16, dv.EINVAL)):
        b = fresh()
        dv.pages_release(b.pool, b.tables, b.i32([1, 0]), b.i32([begin, 0]), b.i32([end, 16]), b.status)
        b.m.release([0], [0], [16])
        b.check(why, copies=False)
    b = fresh()                                       # a table entry that names no page of the pool
    b.tables.table[1, 1] = 60
    dv.pages_fork(b.pool, b.tables, b.i32([1]), b.i32([5]), b.copies, b.status)
    torch.cuda.synchronize()
    assert int(b.status.item()) == dv.ERANGE and b.tables.table[5].tolist()[1] == -1
    b = fresh()                                       # counts that do not agree with the tables
    b.pool.refs[4] = 0
    dv.pages_resize(b.pool, b.tables, b.i32([1]), b.i32([0]), b.copies, b.status)
    torch.cuda.synchronize()
    assert int(b.status.item()) == dv.EINVAL and int(b.pool.refs.min()) == 0


@pytest.mark.parametrize("n_pages", [60, 40000])
@pytest.mark.parametrize("count", [-1, -3, -2 ** 31])
@pytest.mark.parametrize("where", ["behind the used ones", "before their end", "the last page"])
def test_nothing_moves_where_a_count_is_below_zero(dv, n_pages, count, where):
    """A page of such a count that a table names: reported, and all stays as it was; put right, it is compacted."""
    b = Both(dv, n_pages, 16, 8, 30)
    b.resize([0, 1, 2, 3], [33, 200, 480, 5])
    b.resize([1], [0])                                # thirteen holes in front
    if where == "the last page":
        b.m.table[4, 0], b.m.len[4], b.m.refs[n_pages - 1] = n_pages - 1, 9, 1
        b.tables.table[4, 0], b.tables.kv_len[4], b.pool.refs[n_pages - 1] = n_pages - 1, 9, 1
        at = n_pages - 1
    else:
        at = int(b.m.table[2, 29 if where == "behind the used ones" else 0])
    b.pool.refs[at] = count
    refs = b.pool.refs.clone()
    b.copies.count.fill_(5)
    dv.pages_compact(b.pool, b.tables, b.copies, b.status)
    torch.cuda.synchronize()
    assert int(b.status.item()) == dv.EINVAL and int(b.copies.count.item()) == 0
    assert torch.equal(b.pool.refs, refs)
    assert np.array_equal(b.tables.table.cpu().numpy(), b.m.table)
    assert np.array_equal(b.tables.kv_len.cpu().numpy(), b.m.len)
    b.status.zero_()
    b.pool.refs[at] = 1
    b.compact()


def test_captured_calls(dv):
    """A beam search step as a graph: lists and lengths are read anew by every replay."""
    b = Both(dv, 200, 16, 20, 20)
    b.resize([0, 1], [70, 33])
    src, dst, none = b.i32([0, 0, 1]), b.i32([5, 6, 7]), b.i32([0, 0, 0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dv.pages_resize(b.pool, b.tables, dst, none, b.copies, b.status)
        dv.pages_fork(b.pool, b.tables, src, dst, b.copies, b.status)
    for parents in ([0, 0, 1], [1, 1, 1], [0, 1, 0]):
        src.copy_(b.i32(parents))
        graph.replay()
        b.m.resize([5, 6, 7], [0, 0, 0], 200)
        b.m.fork(parents, [5, 6, 7], 200)
        b.check()


def test_calls_behind_one_another(dv):
    """Nothing is looked at between the calls, which start while the ones before them end."""
    r = random.Random(11)
    b = Both(dv, 300, 16, 40, 30)
    todo = []
    for turn in range(60):
        kids = list(range(10 + turn % 20, 20 + turn % 20))
        n = [r.randint(1, 400) for _ in range(3)]
        todo.append((b.i32([0, 1, 2] + kids), b.i32(n + [0] * 10), b.i32([r.randrange(3) for _ in kids]), b.i32(kids)))
    for slots, lens, src, dst in todo:
        dv.pages_resize(b.pool, b.tables, slots, lens, b.copies, b.status)
        dv.pages_fork(b.pool, b.tables, src, dst, b.copies, b.status)
        dv.pages_compact(b.pool, b.tables, b.copies, b.status)
    bad = False
    for slots, lens, src, dst in todo:
        bad |= not b.m.resize(slots.tolist(), lens.tolist(), 300)
        bad |= not b.m.fork(src.tolist(), dst.tolist(), 300)
        b.m.compact(300)
    b.check(dv.ECAP if bad else dv.OK)


def test_as_many_slots_as_there_may_be(dv):
    n = dv.MAX_SLOTS
    b = Both(dv, 100, 128, n, 3)
    b.resize([n - 1, 0, n - 32, 31], [300, 5, 129, 256])
    b.fork([n - 1, n - 32], [n - 2, n - 31])
    b.resize([n - 1], [0])
    b.compact()
    with pytest.raises(dv.DsVitError):
        dv.pages_compact(b.pool, dv.PageTables.empty(n + 1, 3), b.copies)


# ------------------------------------------------------------------ contents

def pages(dv, kind, n, heads, page, dim, seed=0):
    g = torch.Generator().manual_seed(seed)
    shape = (n, heads, page, dim)
    if kind == "bf16":
        return dv.KvCache(*(torch.randn(shape, generator=g).bfloat16().cuda() for _ in range(2)))
    return dv.KvCache(*(torch.randint(0, 256, s, generator=g).to(torch.uint8).cuda()
                        for s in (shape, shape, shape[:3], shape[:3])))


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
@pytest.mark.parametrize("heads,page,dim", [(1, 16, 64), (8, 16, 128), (3, 32, 64), (10, 64, 128), (5, 128, 64)])
@pytest.mark.parametrize("with_bounds", [False, True])
def test_copies_of_pages(dv, kind, heads, page, dim, with_bounds):
    n = 23
    cache = pages(dv, kind, n, heads, page, dim)
    held = [t for t in (cache.k, cache.v, cache.k_exp, cache.v_exp) if t is not None]
    bounds = dv.KeyBounds.empty(cache)
    bounds.hi_lo.copy_(torch.randint(-127, 128, bounds.hi_lo.shape))
    bounds.exp.copy_(torch.randint(0, 256, bounds.exp.shape))
    kept = bounds.hi_lo.clone(), bounds.exp.clone()
    if with_bounds:
        held += [bounds.hi_lo, bounds.exp]
    want = [t.clone() for t in held]
    src, dst = [0, 0, 22, 7, 3], [5, 6, 1, 21, 2]
    for t in want:
        t[dst] = t[src]
    copies = dv.PageCopies(9)
    copies.src.copy_(torch.tensor(src + [9] * 4))
    copies.dst.copy_(torch.tensor(dst + [10] * 4))       # beyond the count: not meant
    copies.count.fill_(5)
    status = dv.cache_copy(cache, copies, bounds if with_bounds else None)
    torch.cuda.synchronize()
    assert int(status.item()) == dv.OK
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(held, want))
    if not with_bounds:
        assert torch.equal(bounds.hi_lo, kept[0]) and torch.equal(bounds.exp, kept[1])


def test_bad_copies_are_left_out(dv):
    cache = pages(dv, "bf16", 6, 2, 16, 64)
    want = cache.k.clone()
    copies = dv.PageCopies(4)
    copies.src.copy_(torch.tensor([0, -1, 6, 1]))
    copies.dst.copy_(torch.tensor([6, 2, 3, 4]))
    for count, why in ((-1, dv.EINVAL), (5, dv.EINVAL), (0, dv.OK)):
        copies.count.fill_(count)
        assert int(dv.cache_copy(cache, copies).item()) == why
        assert torch.equal(cache.k, want)
    copies.count.fill_(4)
    assert int(dv.cache_copy(cache, copies).item()) == dv.ERANGE
    want[4] = want[1]
    assert torch.equal(cache.k, want)


def test_forked_and_compacted_sequences_read_the_same(dv):
    """What a sequence reads back stays the same through a fork and a compaction, and is its own."""
    page, heads, dim = 16, 2, 64
    b = Both(dv, 64, page, 6, 10)
    cache = pages(dv, "bf16", 64, heads, page, dim)
    b.resize([0, 1], [45, 70])

    def chunks(slots, new):
        off = [0]
        for x in new:
            off.append(off[-1] + x)
        at = torch.tensor(slots, device="cuda")
        return dv.Chunks(b.i32(off), b.tables.kv_len[at].contiguous(), b.tables.table[at].contiguous(),
                         max(new)), off[-1]

    g = torch.Generator().manual_seed(1)
    x = torch.randn((115, heads, dim), generator=g).bfloat16().cuda()
    ch, rows = chunks([0, 1], [45, 70])
    dv.cache_write(cache, ch, x, -x)
    b.fork([0, 1, 1], [2, 3, 4])
    dv.cache_copy(cache, b.copies)
    new = torch.randn((3, heads, dim), generator=g).bfloat16().cuda()
    b.resize([2, 3, 4], [46, 71, 71])
    assert b.m.copies == []
    ch, rows = chunks([2, 3, 4], [1, 1, 1])
    dv.cache_write(cache, ch, new, -new)
    b.resize([1], [0])
    b.compact()
    dv.cache_copy(cache, b.copies)
    ch, rows = chunks([0, 2, 3, 4], [45, 46, 71, 71])
    k, v, status = dv.cache_read(cache, ch, rows)
    want = torch.cat([x[:45], x[:45], new[:1], x[45:], new[1:2], x[45:], new[2:]])
    torch.cuda.synchronize()
    assert int(status.item()) == dv.OK and torch.equal(k, want) and torch.equal(v, -want)

"""Argument checks of the calls on pages, without a GPU: refusals come before any CUDA call."""
import ctypes as C

import pytest

P = 4096   # a pointer-like number, 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def dv():
    import __graft_entry__
    __graft_entry__.build()
    import vit_vision_encoder_gb300
    return vit_vision_encoder_gb300


def _make(cls, f, kw):
    f.update(kw)
    return cls(*(f[n] for n, _ in cls._fields_))


def _pool(dv, **kw):
    return _make(dv.PoolArrays, dict(refs=P, n_pages=10, page=16), kw)


def _tables(dv, **kw):
    return _make(dv.TableArrays, dict(table=P, kv_len=P, slots=4, table_cols=5), kw)


def _copies(dv, **kw):
    return _make(dv.CopyArrays, dict(src=P, dst=P, count=P, cap=3), kw)


def _ref(x):
    return None if x is None else C.byref(x)


def _resize(dv, pool, tables, copies, a=P, b=P, c=P, n=0, status=P):
    return dv.lib.ds_vit_pages_resize(_ref(pool), _ref(tables), a, b, n, _ref(copies), status, None)


def _release(dv, pool, tables, copies, a=P, b=P, c=P, n=0, status=P):
    return dv.lib.ds_vit_pages_release(_ref(pool), _ref(tables), a, b, c, n, status, None)


def _fork(dv, pool, tables, copies, a=P, b=P, c=P, n=0, status=P):
    return dv.lib.ds_vit_pages_fork(_ref(pool), _ref(tables), a, b, n, _ref(copies), status, None)


def _compact(dv, pool, tables, copies, a=P, b=P, c=P, n=0, status=P):
    return dv.lib.ds_vit_pages_compact(_ref(pool), _ref(tables), _ref(copies), status, None)


CALLS = [_resize, _release, _fork, _compact]


@pytest.mark.parametrize("call", CALLS)
def test_calls_refused(dv, call):
    """Every call here is refused, so that none is launched."""
    for kw in (dict(refs=None), dict(refs=P + 4), dict(n_pages=0), dict(n_pages=-5), dict(page=8), dict(page=0),
               dict(page=48), dict(page=256)):
        assert call(dv, _pool(dv, **kw), _tables(dv), _copies(dv), n=1) == dv.EINVAL, kw
    for kw in (dict(table=None), dict(table=P + 2), dict(kv_len=None), dict(kv_len=P + 1), dict(slots=0),
               dict(slots=65537), dict(slots=-1), dict(table_cols=0)):
        assert call(dv, _pool(dv), _tables(dv, **kw), _copies(dv), n=1) == dv.EINVAL, kw
    assert call(dv, None, _tables(dv), _copies(dv), n=1) == dv.EINVAL
    assert call(dv, _pool(dv), None, _copies(dv), n=1) == dv.EINVAL
    assert call(dv, _pool(dv), _tables(dv), _copies(dv), n=1, status=None) == dv.EINVAL
    assert call(dv, _pool(dv), _tables(dv), _copies(dv), n=1, status=P + 2) == dv.EINVAL
    assert call(dv, _pool(dv, n_pages=2 ** 31), _tables(dv), _copies(dv), n=1) == dv.ERANGE
    assert call(dv, _pool(dv), _tables(dv, table_cols=2 ** 27), _copies(dv), n=1) == dv.ERANGE


@pytest.mark.parametrize("call", CALLS[:3])
def test_lists_refused(dv, call):
    for kw in (dict(n=0), dict(n=-1), dict(n=1025), dict(n=1, a=None), dict(n=1, b=None), dict(n=1, a=P + 2),
               dict(n=1, b=P + 1)):
        assert call(dv, _pool(dv), _tables(dv), _copies(dv), **kw) == dv.EINVAL, kw
    assert _release(dv, _pool(dv), _tables(dv), None, c=None, n=1) == dv.EINVAL


@pytest.mark.parametrize("call", [_resize, _fork, _compact])
def test_copies_refused(dv, call):
    for kw in (dict(src=None), dict(dst=None), dict(count=None), dict(src=P + 2), dict(dst=P + 1), dict(count=P + 3),
               dict(cap=0), dict(cap=-1)):
        assert call(dv, _pool(dv), _tables(dv), _copies(dv, **kw), n=1) == dv.EINVAL, kw
    assert call(dv, _pool(dv), _tables(dv), None, n=1) == dv.EINVAL


def test_copy_refused(dv):
    f = dict(k=P, v=P, k_exp=None, v_exp=None, n_pages=10, kv_heads=4, page=16, head_dim=128, kind=dv.CACHE_BF16)

    def call(bounds=None, copies=None, status=P, **kw):
        c = dv.Cache(*({**f, **kw}[n] for n, _ in dv.Cache._fields_))
        return dv.lib.ds_vit_cache_copy(C.byref(c), _ref(bounds), _ref(_copies(dv) if copies is None else copies), status,
                                        None)

    for kw in (dict(k=None), dict(v=P + 8), dict(kind=2), dict(kind=dv.CACHE_E4M3), dict(page=8), dict(head_dim=96),
               dict(kv_heads=0), dict(kv_heads=129), dict(n_pages=0), dict(status=None), dict(status=P + 1),
               dict(bounds=dv.BoundArrays(None, P)), dict(bounds=dv.BoundArrays(P, None)),
               dict(bounds=dv.BoundArrays(P + 8, P)), dict(copies=_copies(dv, cap=0)),
               dict(copies=_copies(dv, src=None))):
        assert call(**kw) == dv.EINVAL, kw
    assert call(n_pages=2 ** 40) == dv.ERANGE
    assert dv.lib.ds_vit_cache_copy(None, None, C.byref(_copies(dv)), P, None) == dv.EINVAL


def test_binding_refuses(dv):
    torch = pytest.importorskip("torch")
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)   # noqa: E731
    for make in (lambda: dv.PagePool(i32(4).long(), 16), lambda: dv.PagePool(i32(4), 20),
                 lambda: dv.PagePool(i32(4, 4), 16), lambda: dv.PagePool(i32(8)[::2], 16),
                 lambda: dv.PageTables(i32(3, 4), i32(4)), lambda: dv.PageTables(i32(3), i32(3)),
                 lambda: dv.PageTables(i32(3, 4).long(), i32(3)), lambda: dv.PageTables(i32(4, 3).T, i32(3)),
                 lambda: dv.PageCopies(0, "cpu"), lambda: dv.PageCopies(2 ** 32 + 1, "cpu")):
        with pytest.raises(dv.DsVitError):
            make()
    pool, tables, copies = dv.PagePool(i32(4), 16), dv.PageTables(i32(3, 4), i32(3)), dv.PageCopies(4, "cpu")
    with pytest.raises(dv.DsVitError):                   # not on a GPU
        dv.pages_resize(pool, tables, i32(1), i32(1), copies, i32(1))
    u8 = torch.uint8
    cache = dv.KvCache(*(torch.zeros((3, 2, 16, 64), dtype=torch.bfloat16) for _ in range(2)))
    bounds = dv.KeyBounds.empty(cache)
    assert bounds.of(cache)
    other = dv.KvCache(*(torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16) for _ in range(2)))
    assert not bounds.of(other)
    for args in ((torch.zeros((3, 2, 2, 64), dtype=u8), torch.zeros((3, 2), dtype=u8)),
                 (torch.zeros((3, 2, 3, 64), dtype=torch.int8), torch.zeros((3, 2), dtype=u8)),
                 (torch.zeros((3, 2, 2, 64), dtype=torch.int8), torch.zeros((3, 3), dtype=u8)),
                 (torch.zeros((3, 2, 2, 64), dtype=torch.int8), torch.zeros((3, 2), dtype=torch.int8))):
        with pytest.raises(dv.DsVitError):
            dv.KeyBounds(*args)

"""Argument checks of the bounds, the selection and the attention over blocks, without a GPU:
refusals come before any CUDA call."""
import ctypes as C

import pytest

from test_cache_abi import P, _cache, _chunks


@pytest.fixture(scope="module")
def dv():
    import __graft_entry__
    __graft_entry__.build()
    import vit_vision_encoder_gb300
    return vit_vision_encoder_gb300


def _ref(x):
    return None if x is None else C.byref(x)


GOOD = object()


def _bounds(dv, cache, chunks, b=GOOD, rows=0, status=P):
    return dv.lib.ds_vit_cache_bounds(cache, chunks, _ref(dv.BoundArrays(P, P) if b is GOOD else b), rows, status, None)


def _select(dv, cache, chunks, b=GOOD, q=P, qs=1024, rows=0, heads=8, top=5, first=1, last=2, blocks=P, rs=40, hs=5,
            status=P):
    return dv.lib.ds_vit_cache_select(cache, chunks, _ref(dv.BoundArrays(P, P) if b is GOOD else b), q, qs, rows, heads,
                                      top, first, last, blocks, rs, max(hs, top if hs == 5 else 0), status, None)


def _attend(dv, cache, chunks, q=P, qs=1024, rows=0, heads=8, scale=0.1, blocks=P, rs=40, hs=5, top=5, out=2 * P,
            os_=1024, status=P):
    return dv.lib.ds_vit_cache_attention_blocks(cache, chunks, q, qs, rows, heads, scale, blocks, rs, hs, top, out, os_,
                                                status, None)


@pytest.mark.parametrize("call", [_bounds, _select, _attend])
def test_caches_and_chunks_refused(dv, call):
    ca, ch = C.byref(_cache(dv)), C.byref(_chunks(dv))
    assert call(dv, ca, ch) == dv.OK
    assert call(dv, None, ch) == dv.EINVAL and call(dv, ca, None) == dv.EINVAL
    for kw in (dict(k=None), dict(v=P + 8), dict(kind=2), dict(kind=dv.CACHE_E4M3), dict(page=24), dict(head_dim=72),
               dict(kv_heads=0), dict(n_pages=0)):
        assert call(dv, C.byref(_cache(dv, **kw)), ch) == dv.EINVAL, kw
    for kw in (dict(row_off=None), dict(kv_len=P + 1), dict(table=P + 2), dict(n=0), dict(n=1025), dict(max_rows=0)):
        assert call(dv, ca, C.byref(_chunks(dv, **kw))) == dv.EINVAL, kw
    assert call(dv, ca, ch, rows=-1) == dv.EINVAL
    assert call(dv, ca, ch, rows=2 ** 30) == dv.ERANGE
    for kw in (dict(status=None), dict(status=P + 2)):
        assert call(dv, ca, ch, **kw) == dv.EINVAL


@pytest.mark.parametrize("call", [_bounds, _select])
def test_bounds_refused(dv, call):
    ca, ch = C.byref(_cache(dv)), C.byref(_chunks(dv))
    for b in (None, dv.BoundArrays(None, P), dv.BoundArrays(P, None), dv.BoundArrays(P + 8, P)):
        assert call(dv, ca, ch, b=b) == dv.EINVAL


def test_select_refused(dv):
    ca, ch = C.byref(_cache(dv)), C.byref(_chunks(dv))
    for kw in (dict(q=None), dict(q=P + 8), dict(qs=1016), dict(qs=1028), dict(heads=0), dict(heads=6),
               dict(heads=4 * 129), dict(top=2), dict(top=0), dict(top=4097), dict(first=-1), dict(last=0),
               dict(last=-3), dict(first=2 ** 31 - 1, last=2 ** 31 - 1), dict(blocks=None), dict(blocks=P + 2), dict(hs=4),
               dict(rows=2, rs=3)):
        assert _select(dv, ca, ch, **kw) == dv.EINVAL, kw
    assert _select(dv, ca, ch, top=3) == dv.OK and _select(dv, ca, ch, top=4096) == dv.OK
    wide = C.byref(_chunks(dv, table_cols=dv.SELECT_MAX_COLS))
    assert _select(dv, ca, wide) == dv.OK
    assert _select(dv, ca, C.byref(_chunks(dv, table_cols=dv.SELECT_MAX_COLS + 1))) == dv.ERANGE
    assert _select(dv, ca, ch, rows=2 ** 29) == dv.ERANGE                       # 4 K/V heads


def test_attention_refused(dv):
    ca, ch = C.byref(_cache(dv)), C.byref(_chunks(dv))
    for kw in (dict(q=None), dict(out=None), dict(q=P + 8), dict(out=P + 8), dict(qs=1016), dict(os_=1020),
               dict(heads=0), dict(heads=6), dict(heads=4 * 129), dict(scale=0.0), dict(scale=-1.0),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(blocks=None), dict(blocks=P + 2), dict(hs=4),
               dict(rows=2, rs=3), dict(top=0),
               dict(top=-1), dict(top=4097)):
        assert _attend(dv, ca, ch, **kw) == dv.EINVAL, kw
    assert _attend(dv, ca, ch, rows=2 ** 28) == dv.ERANGE                       # 8 heads


def test_binding_refuses(dv):
    """Tensors that the binding can tell are wrong (none of them on a GPU: nothing is called)."""
    torch = pytest.importorskip("torch")
    z = lambda s, t=torch.bfloat16: torch.zeros(s, dtype=t)   # noqa: E731
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32)        # noqa: E731
    cache = dv.KvCache(z((3, 2, 16, 64)), z((3, 2, 16, 64)))
    chunks = dv.Chunks(i32(2), i32(1), i32(1, 3), 1)
    bounds = dv.KeyBounds.empty(cache)
    for call in (lambda: dv.cache_bounds(cache, chunks, bounds, 1), lambda: dv.cache_select(cache, chunks, bounds, z((1, 4, 64)), 2),
                 lambda: dv.cache_attention_blocks(cache, chunks, z((1, 4, 64)), i32(1, 2, 2))):
        with pytest.raises(dv.DsVitError):
            call()
    lists = dv._block_lists
    assert lists(i32(5, 2, 7), 5, 2, -1, "") == (7, 14, 7)
    assert lists(i32(2, 5, 9).transpose(0, 1)[..., 1:8], 5, 2, -1, "") == (7, 9, 45)
    for t in (i32(5, 2, 7).long(), i32(5, 3, 7), i32(4, 2, 7), i32(5, 2), i32(5, 7, 2).transpose(1, 2)):
        with pytest.raises(dv.DsVitError):
            lists(t, 5, 2, -1, "")

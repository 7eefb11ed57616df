"""The paged-cache entry points' argument checks, without a GPU: every refusal
comes before any CUDA call, so made-up pointers are never followed."""
import ctypes as C
import threading

import pytest


@pytest.fixture(scope="module")
def dv():
    import __graft_entry__
    __graft_entry__.build()
    import vit_vision_encoder_gb300
    return vit_vision_encoder_gb300


P = 4096   # a pointer-like number, 16-byte aligned, never dereferenced


def _cache(dv, **kw):
    f = dict(k=P, v=P, k_exp=None, v_exp=None, n_pages=10, kv_heads=4, page=16, head_dim=128, kind=dv.CACHE_BF16)
    f.update(kw)
    return dv.Cache(*(f[n] for n, _ in dv.Cache._fields_))


def _chunks(dv, **kw):
    f = dict(row_off=P, kv_len=P, table=P, n=2, table_cols=5, max_rows=3)
    f.update(kw)
    return dv.ChunkArrays(*(f[n] for n, _ in dv.ChunkArrays._fields_))


def _write(dv, cache, chunks, k=P, ks=512, v=P, vs=512, rows=0, status=P):
    return dv.lib.ds_vit_cache_write(cache, chunks, k, ks, v, vs, rows, status, None)


def _read(dv, cache, chunks, k=P, ks=512, v=P, vs=512, rows=0, status=P):
    return dv.lib.ds_vit_cache_read(cache, chunks, k, ks, v, vs, rows, status, None)


def _attend(dv, cache, chunks, q=P, qs=1024, rows=0, heads=8, scale=0.1, window=0, sinks=0, out=2 * P, os_=1024,
            ws=P, ws_bytes=1 << 40, status=P):
    return dv.lib.ds_vit_cache_attention(cache, chunks, q, qs, rows, heads, scale, window, sinks, out, os_, ws,
                                         ws_bytes, status, None)


CALLS = [_write, _read, _attend]


@pytest.mark.parametrize("call", CALLS)
def test_no_rows_is_no_work(dv, call):
    assert call(dv, C.byref(_cache(dv)), C.byref(_chunks(dv))) == dv.OK


@pytest.mark.parametrize("call", CALLS)
def test_caches_refused(dv, call):
    ch = C.byref(_chunks(dv))
    assert call(dv, None, ch) == dv.EINVAL
    for kw in (dict(k=None), dict(v=None), dict(k=P + 8), dict(v=P + 2), dict(kind=2), dict(kind=-1),
               dict(kind=dv.CACHE_E4M3), dict(kind=dv.CACHE_E4M3, k_exp=C.cast(P, C.c_void_p)), dict(page=8),
               dict(page=24), dict(page=256), dict(page=0), dict(page=-16), dict(head_dim=72), dict(head_dim=256),
               dict(kv_heads=0), dict(kv_heads=129), dict(n_pages=0), dict(n_pages=-1)):
        assert call(dv, C.byref(_cache(dv, **kw)), ch) == dv.EINVAL, kw
    for n_pages, ok in ((2 ** 31 // 64 - 1, True), (2 ** 31 // 64, False), (2 ** 40, False)):
        assert call(dv, C.byref(_cache(dv, n_pages=n_pages)), ch) == (dv.OK if ok else dv.ERANGE)


@pytest.mark.parametrize("call", CALLS)
def test_chunks_refused(dv, call):
    ca = C.byref(_cache(dv))
    assert call(dv, ca, None) == dv.EINVAL
    for kw in (dict(row_off=None), dict(kv_len=None), dict(table=None), dict(row_off=P + 2), dict(kv_len=P + 1),
               dict(table=P + 2), dict(n=0), dict(n=1025), dict(table_cols=0), dict(max_rows=0)):
        assert call(dv, ca, C.byref(_chunks(dv, **kw))) == dv.EINVAL, kw
    assert call(dv, ca, C.byref(_chunks(dv, n=1024))) == dv.OK
    assert call(dv, ca, C.byref(_chunks(dv, table_cols=2 ** 27))) == dv.ERANGE
    assert call(dv, ca, C.byref(_chunks(dv)), rows=-1) == dv.EINVAL
    assert call(dv, ca, C.byref(_chunks(dv)), rows=2 ** 30) == dv.ERANGE


@pytest.mark.parametrize("call", [_write, _read])
def test_rows_refused(dv, call):
    ca, ch = C.byref(_cache(dv)), C.byref(_chunks(dv))
    for kw in (dict(k=None), dict(v=None), dict(k=P + 8), dict(v=P + 4), dict(ks=511), dict(ks=504), dict(vs=0),
               dict(vs=516), dict(status=None), dict(status=P + 2)):
        assert call(dv, ca, ch, **kw) == dv.EINVAL, kw
    assert call(dv, ca, ch, ks=520, vs=4096) == dv.OK


def test_attention_refused(dv):
    ca, ch = C.byref(_cache(dv)), C.byref(_chunks(dv))
    for kw in (dict(q=None), dict(out=None), dict(ws=None), dict(q=P + 8), dict(out=P + 8), dict(ws=P + 8),
               dict(qs=1016), dict(os_=1020), dict(heads=0), dict(heads=6), dict(heads=4 * 129), dict(scale=0.0),
               dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(window=-1), dict(sinks=-1),
               dict(status=None)):
        assert _attend(dv, ca, ch, **kw) == dv.EINVAL, kw
    assert _attend(dv, ca, ch, ws_bytes=0) == dv.ECAP
    n = C.c_size_t(0)
    size = dv.lib.ds_vit_cache_attention_workspace_bytes
    assert size(ca, ch, 8, None) == dv.EINVAL
    assert size(ca, ch, 7, C.byref(n)) == dv.EINVAL
    assert size(None, ch, 8, C.byref(n)) == dv.EINVAL
    assert size(ca, ch, 8, C.byref(n)) == dv.OK and n.value > 0
    assert _attend(dv, ca, ch, ws_bytes=n.value) == dv.OK
    assert _attend(dv, ca, ch, ws_bytes=n.value - 1) == dv.ECAP


def test_binding_refuses_other_tensors(dv):
    """The binding checks what the C call cannot see: types, shapes, strides."""
    torch = pytest.importorskip("torch")
    z = lambda shape, t=torch.bfloat16: torch.zeros(shape, dtype=t)   # noqa: E731
    pages = (3, 2, 16, 64)
    cache = dv.KvCache(z(pages), z(pages))
    assert (cache.c.n_pages, cache.c.kv_heads, cache.c.page, cache.c.head_dim) == pages
    u8 = torch.uint8
    quant = dv.KvCache(z(pages, u8), z(pages, u8), z(pages[:3], u8), z(pages[:3], u8))
    assert quant.c.kind == dv.CACHE_E4M3
    for args in ((z(pages), z(pages, torch.float16)), (z(pages, torch.float16), z(pages, torch.float16)),
                 (z(pages, u8), z(pages, u8)), (z(pages, u8), z(pages, u8), z(pages[:3], u8), z((3, 2, 15), u8)),
                 (z(pages), z((3, 2, 16, 32))), (z(pages).transpose(0, 1), z(pages).transpose(0, 1))):
        with pytest.raises(dv.DsVitError):
            dv.KvCache(*args)
    i32 = torch.int32
    ch = dv.Chunks(z(3, i32), z(2, i32), z((2, 4), i32), 1)
    for args in ((z(2, i32), z(2, i32), z((2, 4), i32)), (z(3, torch.int64), z(2, i32), z((2, 4), i32)),
                 (z(3, i32), z(2, i32), z((1, 4), i32)), (z(3, i32), z(2, i32), z((2, 8), i32)[:, ::2])):
        with pytest.raises(dv.DsVitError):
            dv.Chunks(*args, 1)
    st = z(1, i32)
    for k, v in ((z((5, 2, 64), torch.float32), z((5, 2, 64), torch.float32)), (z((5, 3, 64)), z((5, 3, 64))),
                 (z((5, 2, 64)), z((4, 2, 64))), (z((5, 64, 2)).transpose(1, 2), z((5, 2, 64))),
                 (z((2, 5, 64)).transpose(0, 1), z((5, 2, 64)))):
        with pytest.raises(dv.DsVitError):
            dv.cache_write(cache, ch, k, v, status=st)
    with pytest.raises(dv.DsVitError):
        dv.cache_attention(cache, ch, z((5, 4, 64)), out=z((5, 2, 64)), status=st)
    with pytest.raises(dv.DsVitError):
        dv.cache_read(cache, ch, 5, out=(z((4, 2, 64)), z((4, 2, 64))), status=st)


def test_each_thread_has_a_workspace(dv, monkeypatch):
    """Threads that share a stream do not share the workspace kept for it: a call makes two
    launches, and another thread's may come between them."""
    torch = pytest.importorskip("torch")
    z = lambda shape, t=torch.bfloat16: torch.zeros(shape, dtype=t)   # noqa: E731
    cache = dv.KvCache(z((3, 2, 16, 64)), z((3, 2, 16, 64)))
    ch = dv.Chunks(z(3, torch.int32), z(2, torch.int32), z((2, 4), torch.int32), 1)
    monkeypatch.setattr(dv, "_capturing", lambda: False)
    got, both = {}, threading.Barrier(3, timeout=60)

    def thread(name):
        a = dv._workspace(cache, ch, 4, 77)
        got[name] = a, dv._workspace(cache, ch, 4, 77), dv._workspace(cache, ch, 4, 78)
        both.wait()                     # all are alive at once

    threads = [threading.Thread(target=thread, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    both.wait()
    for t in threads:
        t.join()
    mine = dv._workspace(cache, ch, 4, 77)
    places = [mine.data_ptr()]
    for a, again, other in got.values():
        assert a.data_ptr() == again.data_ptr()
        places += [a.data_ptr(), other.data_ptr()]
    assert len(set(places)) == 5


@pytest.mark.parametrize("max_rows", [2 ** 31, 2 ** 32, 2 ** 32 + 3, -1])
def test_counts_past_32_bits_refused(dv, max_rows):
    """ctypes would hand on what is left modulo 2^32."""
    torch = pytest.importorskip("torch")
    z = lambda shape: torch.zeros(shape, dtype=torch.int32)   # noqa: E731
    with pytest.raises(dv.DsVitError):
        dv.Chunks(z(3), z(2), z((2, 4)), max_rows)
    assert dv.Chunks(z(3), z(2), z((2, 4)), 2 ** 31 - 1).c.max_rows == 2 ** 31 - 1

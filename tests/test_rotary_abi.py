"""Argument checks of the norms and rotation without a GPU (refusals come before any CUDA
call), and the table that ds_vit_rotary_init makes."""
import ctypes as C
import random
from fractions import Fraction

import pytest

P = 4096   # a pointer-like number, 16-byte aligned, never dereferenced


@pytest.fixture(scope="module")
def dv():
    import __graft_entry__
    __graft_entry__.build()
    import vit_vision_encoder_gb300
    return vit_vision_encoder_gb300


def _init(dv, head_dim=128, theta=1e4, inv=None, axes=1, sections=None, interleaved=0, pairing=1, out=True):
    r = dv.RotaryTable()
    s = None if sections is None else (C.c_int32 * 3)(*sections)
    f = None if inv is None else (C.c_double * len(inv))(*inv)
    return dv.lib.ds_vit_rotary_init(head_dim, theta, f, axes, s, interleaved, pairing, C.byref(r) if out else None), r


def test_tables_refused(dv):
    inf, nan = float("inf"), float("nan")
    for kw in (dict(head_dim=72), dict(head_dim=0), dict(theta=1.0), dict(theta=-5.0), dict(theta=inf), dict(theta=nan),
               dict(axes=2), dict(axes=0), dict(axes=3), dict(axes=3, sections=(24, 20, 21)), dict(pairing=0),
               dict(axes=3, sections=(104, -20, -20)), dict(pairing=3), dict(inv=[1.0] * 63 + [0.0]),
               dict(inv=[nan] + [1.0] * 63), dict(inv=[1.0] * 63 + [inf]), dict(out=False),
               dict(axes=3, sections=(10, 22, 32), interleaved=1), dict(axes=3, sections=(20, 22, 22), interleaved=1)):
        assert _init(dv, **kw)[0] == dv.EINVAL, kw
    assert _init(dv, theta=-1.0, inv=[1.0] * 64)[0] == dv.OK
    assert _init(dv, axes=3, sections=(21, 21, 22), interleaved=1)[0] == dv.EINVAL      # 2, 5, .. 62: 21 pairs
    assert _init(dv, axes=3, sections=(22, 21, 21), interleaved=1)[0] == dv.OK
    assert _init(dv, axes=3, sections=(10, 22, 32))[0] == dv.OK


def test_tables(dv):
    rc, r = _init(dv, 64, 1e6, axes=3, sections=(12, 10, 10), interleaved=1, pairing=2)
    assert rc == dv.OK and (r.head_dim, r.axes, r.pairing) == (64, 3, 2)
    assert list(r.axis)[:32] == [i % 3 if i % 3 and i < 30 else 0 for i in range(32)]
    assert [list(r.axis)[:32].count(a) for a in range(3)] == [12, 10, 10]
    two_pi = Fraction(314159265358979323846264338327950288, 10 ** 35) * 2
    for inv in ([1.0, 0.25, 6.5, 1e-9] * 16, [2.0 ** -i for i in range(64)]):
        rc, r = _init(dv, inv=inv)
        assert rc == dv.OK
        for f, t in zip(inv, r.turn):
            want = (Fraction(f) / two_pi) % 1
            assert abs(Fraction(t, 2 ** 64) - want) <= Fraction(1, 2 ** 55) * max(1, int(f) + 1)
    rc, r = _init(dv, axes=3, sections=(24, 20, 20))
    assert list(r.axis) == [0] * 24 + [1] * 20 + [2] * 20


def _pi(bits):
    """pi in units of 2^-bits, by 16 atan(1/5) - 4 atan(1/239)."""
    def atan_of(x):
        term = total = (1 << bits) // x
        n = 1
        while term:
            term //= x * x
            n += 2
            total += -(term // n) if n % 4 == 3 else term // n
        return total
    return 16 * atan_of(5) - 4 * atan_of(239)


def test_turns_of_given_frequencies(dv):
    """Right to 2^-63 turns a position up to frequencies of 2^64, over a radian a position as well as under."""
    two_pi = Fraction(_pi(400), 2 ** 399)
    r = random.Random(3)
    given = [0.99, 1.0, 1.3, 6.283185307179586, 6.5, 100.0, 12345.678, 1e6 + 0.1, 2.0 ** 31 - 0.5, 1e15 + 0.5, 1.7e16, 1e19,
             2.0 ** 64, 1e-9, 1e-18, 2.0 ** -62, 2.0 ** -64, 1e-30, 1e-300, 5e-324]
    given += [r.uniform(1, 2) * 2.0 ** r.randint(-70, 63) for _ in range(64 * 20 - len(given))]
    for i in range(0, len(given), 64):
        rc, t = _init(dv, inv=given[i:i + 64])
        assert rc == dv.OK
        for f, turn in zip(given[i:i + 64], t.turn):
            off = (Fraction(turn, 2 ** 64) - Fraction(f) / two_pi) % 1
            assert min(off, 1 - off) <= Fraction(1, 2 ** 63), f
    assert _init(dv, inv=[1.7e308] * 64)[0] == dv.OK


@pytest.mark.parametrize("head_dim", [64, 128])
@pytest.mark.parametrize("theta", [1.0000001, 2.0, 1e4, 5e5, 1e6, 1e7, 1e300])
def test_turns_of_a_theta(dv, head_dim, theta):
    """Right to 2^-55 turns a position: those of theta^(-2i/d) as a double, which is at most 1."""
    two_pi = Fraction(_pi(400), 2 ** 399)
    rc, t = _init(dv, head_dim, theta)
    assert rc == dv.OK
    for i, turn in zip(range(head_dim // 2), t.turn):
        # theta^(-2i/d) by its head_dim/2-th power: what lies between a step of 2^-55 turns to either side.
        lo, hi = ((Fraction(turn, 2 ** 64) + d) * two_pi for d in (Fraction(-1, 2 ** 55), Fraction(1, 2 ** 55)))
        want = 1 / Fraction(theta) ** i
        assert (max(lo, 0) ** (head_dim // 2) <= want <= hi ** (head_dim // 2)), i


def _call(dv, r, q=P, qs=1024, heads=8, k=P, ks=256, kv=2, rows=0, pos=P, ps=100, qn=None, kn=None, eps=1e-6, qo=P,
          qos=1024, ko=P, kos=256):
    return dv.lib.ds_vit_qk_norm_rope(r, q, qs, heads, k, ks, kv, rows, pos, ps, qn, kn, eps, qo, qos, ko, kos, None)


def test_calls_refused(dv):
    _, r = _init(dv)
    ref = C.byref(r)
    assert _call(dv, ref) == dv.OK
    assert _call(dv, ref, qs=1032, kos=4096, eps=-1.0, ps=0) == dv.OK        # no norm, one axis
    nan = float("nan")
    for kw in (dict(q=None), dict(k=None), dict(qo=None), dict(ko=None), dict(pos=None), dict(q=P + 8), dict(k=P + 2),
               dict(qo=P + 8), dict(ko=P + 4), dict(pos=P + 2), dict(qn=P + 8), dict(kn=P + 2), dict(qs=1016),
               dict(qs=1028), dict(ks=255), dict(qos=0), dict(kos=-256), dict(heads=0), dict(heads=16385), dict(kv=0),
               dict(kv=129), dict(rows=-1), dict(qn=P, eps=0.0), dict(kn=P, eps=nan), dict(qn=P, eps=-1e-6),
               dict(qn=P, eps=float("inf"))):
        assert _call(dv, ref, **kw) == dv.EINVAL, kw
    assert _call(dv, None) == dv.EINVAL
    assert _call(dv, ref, rows=2 ** 30) == dv.ERANGE
    _, three = _init(dv, axes=3, sections=(24, 20, 20))
    assert _call(dv, C.byref(three), rows=101, ps=100) == dv.EINVAL
    for field, value in (("head_dim", 96), ("axes", 2), ("axes", 0), ("pairing", 0)):
        _, bad = _init(dv)
        setattr(bad, field, value)
        assert _call(dv, C.byref(bad)) == dv.EINVAL, field
    _, bad = _init(dv)
    bad.axis[5] = 1
    assert _call(dv, C.byref(bad)) == dv.EINVAL


def test_binding_refuses(dv):
    torch = pytest.importorskip("torch")
    for kw in (dict(pairing="other"), dict(head_dim=96), dict(sections=(60,)), dict(sections=(1, 2)), dict(theta=0.5),
               dict(inv_freq=[1.0] * 63), dict(sections=(24, 20, 2 ** 32 + 20)), dict(head_dim=2 ** 32 + 128)):
        with pytest.raises(dv.DsVitError):
            dv.Rotary(**{"head_dim": 128, **kw})
    r = dv.Rotary(128)
    x = torch.zeros((2, 4, 128), dtype=torch.bfloat16)      # not on a GPU
    with pytest.raises(dv.DsVitError):
        dv.qk_norm_rope(r, x, x, torch.zeros(2, dtype=torch.int32))

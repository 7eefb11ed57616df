"""Norms of queries and keys and their rotation by position on the GPU, against the
formula in 64 bits: head layouts, lengths, strides, axes, pairings, far and negative
positions, in place, streams and captured graphs."""
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


def f64(t):
    return t.detach().cpu().double().numpy()


def axis_of(i, dim, sections, interleaved):
    if len(sections) == 1:
        return 0
    if interleaved:
        return i % 3 if i % 3 and i < 3 * sections[i % 3] else 0
    return 0 if i < sections[0] else 1 if i < sections[0] + sections[1] else 2


def rotate64(x, pos, freq, sections, interleaved, pairing, g, eps):
    """(reference, tolerance) of rows x [rows, heads, dim] (float64).

    Tolerance of one output: its rounding to bf16 (2^-8 of it), and of its pair's
    normed values 2^-19 for fp32: the sum of squares' 20 additions in a row (2^-20.7, half
    of it in the root), rsqrt (2^-22.4), three products, the angle's rounding to 24 bits (pi 2^-25)
    and sincospi (2^-23) together stay under 2^-20.  The angle itself is right to
    2^-55 turns a position, the reference's to 2^-52 of it."""
    rows, heads, dim = x.shape
    n, half = x, dim // 2
    if g is not None:
        n = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * g
    y, tol = np.empty_like(n), np.empty_like(n)
    for i in range(half):
        a, b = (i, i + half) if pairing == "half_vector" else (2 * i, 2 * i + 1)
        p = pos[axis_of(i, dim, sections, interleaved)].astype(np.float64)[:, None]
        t = p * freq[i]
        c, s = np.cos(t), np.sin(t)
        y[..., a] = n[..., a] * c - n[..., b] * s
        y[..., b] = n[..., b] * c + n[..., a] * s
        size = np.abs(n[..., a]) + np.abs(n[..., b])
        off = 2.0 ** -19 + np.abs(p) * (2 * math.pi * 2.0 ** -55 + freq[i] * 2.0 ** -52)
        tol[..., a] = tol[..., b] = size * off
    return y, tol + 2.0 ** -8 * np.abs(y)


def sections_of(dim, axes):
    half = dim // 2
    side = half * 5 // 16
    return (half - 2 * side, side, side) if axes == 3 else (half,)


def case(dv, rows, heads, kv_heads, dim, axes=1, interleaved=False, pairing="half_vector", norms=(True, True), far=5000,
         theta=1000000.0, inv_freq=None, eps=1e-6, wide=0, out="new", positions=None, scale=1.0, seed=0):
    g = torch.Generator().manual_seed(seed)
    qkv = (torch.randn((rows, heads + 2 * kv_heads + wide, dim), generator=g) * scale).bfloat16().cuda()
    q, k = qkv[:, :heads], qkv[:, heads:heads + kv_heads]
    before = qkv.clone()
    pos = torch.randint(0, far, (axes, rows), generator=g).int() if positions is None else positions
    weights = [(1 + 0.3 * torch.randn(dim, generator=g)).bfloat16().cuda() if on else None for on in norms]
    sections = sections_of(dim, axes)
    rotary = dv.Rotary(dim, theta, sections, interleaved, pairing, inv_freq)
    freq = ([theta ** (-2 * i / dim) for i in range(dim // 2)] if inv_freq is None else list(inv_freq))
    refs = [rotate64(f64(x), pos.numpy().reshape(axes, rows), freq, sections, interleaved, pairing,
                     None if w is None else f64(w), eps) for x, w in zip((q, k), weights)]
    out = (q, k) if out == "in place" else None
    got = dv.qk_norm_rope(rotary, q, k, pos.cuda(), *weights, eps, out=out)
    torch.cuda.synchronize()
    for x, (ref, tol) in zip(got, refs):
        err = np.abs(f64(x) - ref)
        bad = ~(err <= tol)
        assert not bad.any(), (bad.sum(), np.nanmax(err / np.maximum(tol, 1e-300)), np.argwhere(bad)[:4].tolist())
    # What lies beside the heads (values, and the inputs if not in place) is as it was.
    kept = heads + kv_heads if out is not None else 0
    assert torch.equal(qkv[:, kept:].view(torch.int16), before[:, kept:].view(torch.int16))
    return got


@pytest.mark.parametrize("rows", [1, 2, 5, 48, 333, 6000])
@pytest.mark.parametrize("heads,kv_heads,dim", [(40, 8, 128), (16, 4, 64), (7, 1, 128), (1, 1, 64), (3, 3, 64)])
def test_rows_and_heads(dv, rows, heads, kv_heads, dim):
    case(dv, rows if rows < 6000 or heads == 40 else 700, heads, kv_heads, dim, axes=3, interleaved=True, seed=rows)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("pairing", ["half_vector", "adjacent"])
@pytest.mark.parametrize("axes,interleaved", [(1, False), (3, False), (3, True)])
def test_pairs_and_axes(dv, dim, pairing, axes, interleaved):
    case(dv, 37, 10, 2, dim, axes, interleaved, pairing, seed=3)


@pytest.mark.parametrize("norms", [(True, False), (False, True), (False, False)])
def test_a_norm_left_out(dv, norms):
    case(dv, 11, 8, 2, 128, norms=norms, eps=1e-5)


@pytest.mark.parametrize("pairing", ["half_vector", "adjacent"])
@pytest.mark.parametrize("rows", [3, 5000])
def test_in_place(dv, pairing, rows):
    case(dv, rows, 12, 4, 64, 3, True, pairing, wide=1, out="in place")


def test_far_and_negative_positions(dv):
    pos = torch.tensor([[0, 1, -1, 1000003, -1000003, 2 ** 31 - 1, -2 ** 31, 123456789]], dtype=torch.int32)
    for pairing in ("half_vector", "adjacent"):
        case(dv, 8, 5, 1, 128, pairing=pairing, positions=pos, theta=500000.0)


def test_one_axis_as_a_vector_and_scaled_frequencies(dv):
    inv = [0.37 / (1.3 ** i) + 1e-3 * i for i in range(32)]
    case(dv, 9, 4, 2, 64, inv_freq=inv, positions=torch.arange(900, 909, dtype=torch.int32))
    case(dv, 9, 4, 2, 64, inv_freq=[3.5 * x for x in inv])        # over a radian a position


@pytest.mark.parametrize("scale", [1e-20, 1e-4, 1e4, 1e15])
def test_magnitudes(dv, scale):
    case(dv, 6, 4, 2, 128, scale=scale, eps=1e-6)


def test_rows_of_zeros_and_not_finite_ones(dv):
    q = torch.ones((4, 2, 64), dtype=torch.bfloat16, device="cuda")
    q[0] = 0
    q[1, 0, 5] = math.inf
    q[2, 1, 7] = math.nan
    w = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    r = dv.Rotary(64)
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    y, k = dv.qk_norm_rope(r, q, q, pos, w, w)
    assert torch.equal(y, k) or torch.isnan(y).any()
    assert (y[0] == 0).all()
    assert not torch.isfinite(y[1, 0]).all() and torch.isfinite(y[1, 1]).all()
    assert torch.isnan(y[2, 1]).all() and torch.isfinite(y[2, 0]).all() and torch.isfinite(y[3]).all()


@pytest.mark.parametrize("pairing", ["half_vector", "adjacent"])
@pytest.mark.parametrize("rows", [4, 700])
def test_queries_and_keys_are_treated_alike(dv, pairing, rows):
    """The same heads as queries and as keys give the same bits, whatever is in other heads, zeros and NaN among them."""
    g = torch.Generator().manual_seed(rows)
    x = torch.randn((rows, 12, 64), generator=g).bfloat16().cuda()
    x[0] = 0
    x[1, 0, 5] = math.inf
    x[2, 1, 7] = math.nan
    w = (1 + 0.3 * torch.randn(64, generator=g)).bfloat16().cuda()
    r = dv.Rotary(64, pairing=pairing)
    pos = torch.arange(rows, dtype=torch.int32, device="cuda")
    y, k = dv.qk_norm_rope(r, x, x[:, :5], pos, w, w)
    torch.cuda.synchronize()
    assert torch.equal(y[:, :5].view(torch.int16), k.view(torch.int16))
    assert torch.isfinite(y[3:]).all() and torch.isfinite(y[1, 1:]).all() and torch.isnan(k[2, 1]).all()


def test_positions_of_an_image_prompt(dv):
    """The three axes that the layout of an image span gives, text before it."""
    span, delta = dv.qwen_layout(5, 7, 20)
    text = np.tile(np.arange(20, dtype=np.int32), (3, 1))
    pos = torch.from_numpy(np.concatenate([text, span], 1).astype(np.int32))
    case(dv, pos.shape[1], 8, 2, 128, 3, True, positions=pos)
    case(dv, pos.shape[1], 8, 2, 128, 3, False, positions=pos)


def test_strided_positions_and_no_rows(dv):
    r = dv.Rotary(128, sections=(24, 20, 20))
    q = torch.randn((10, 4, 128), device="cuda").bfloat16()
    wide = torch.randint(0, 1000, (3, 50), device="cuda").int()
    a = dv.qk_norm_rope(r, q, q[:, :2], wide[:, 7:17])
    b = dv.qk_norm_rope(r, q, q[:, :2], wide[:, 7:17].contiguous())
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    got = dv.qk_norm_rope(r, q[:0], q[:0, :2], wide[:, :0])
    assert got[0].shape == (0, 4, 128) and got[1].shape == (0, 2, 128)


def test_streams_and_a_captured_graph(dv):
    r = dv.Rotary(128, sections=(24, 20, 20), interleaved=True)
    q = torch.randn((200, 10, 128), device="cuda").bfloat16()
    k = torch.randn((200, 2, 128), device="cuda").bfloat16()
    pos = torch.randint(0, 1000, (3, 200), device="cuda").int()
    want = dv.qk_norm_rope(r, q, k, pos)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = dv.qk_norm_rope(r, q, k, pos)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want))
    out = tuple(torch.zeros_like(x) for x in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dv.qk_norm_rope(r, q, k, pos, out=out)
    pos += 5                                      # replays read positions anew
    q.neg_()
    graph.replay()
    want = dv.qk_norm_rope(r, q, k, pos)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(out, want))

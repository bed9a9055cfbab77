"""tq_rope: rotary positions of queries and keys, against the definition in 64 bits."""
import ctypes
import math

import numpy as np
import pytest

import kv_cache_vector_08_b200 as tq

torch = pytest.importorskip("torch")
gpu = pytest.mark.gpu
DEV = torch.device("cuda", 0)


# ------------------------------------------------------------------ host
def test_frequencies_without_scaling_and_linear():
    f, m = tq.rope_frequencies(64, 10000.0)
    assert m == 1.0 and np.allclose(f, 10000.0 ** (-np.arange(0, 64, 2) / 64), rtol=1e-14)
    g, m = tq.rope_frequencies(64, 10000.0, "linear", factor=4.0)
    assert m == 1.0 and np.allclose(g, f / 4, rtol=1e-14)


def test_frequencies_ntk_keeps_the_first_pair_and_interpolates_the_last():
    f, _ = tq.rope_frequencies(128, 10000.0)
    g, m = tq.rope_frequencies(128, 10000.0, "ntk", factor=8.0)
    assert m == 1.0 and g[0] == 1.0 and math.isclose(g[-1], f[-1] / 8.0, rel_tol=1e-12)


def test_frequencies_bands_and_yarn_at_their_ends():
    f, _ = tq.rope_frequencies(128, 500000.0)
    g, m = tq.rope_frequencies(128, 500000.0, "bands", factor=8.0, original_len=8192, low=1.0, high=4.0)
    turns = 8192 * f / (2 * math.pi)
    assert m == 1.0 and np.array_equal(g[turns >= 4], f[turns >= 4])
    assert np.allclose(g[turns <= 1], f[turns <= 1] / 8, rtol=1e-14)
    mid = (turns > 1) & (turns < 4)
    w = (turns[mid] - 1) / 3
    assert mid.any() and np.allclose(g[mid], f[mid] * (w + (1 - w) / 8), rtol=1e-13)
    f, _ = tq.rope_frequencies(64, 10000.0)
    g, m = tq.rope_frequencies(64, 10000.0, "yarn", factor=32.0, original_len=4096)
    assert math.isclose(m, 0.1 * math.log(32.0) + 1.0)
    assert g[0] == f[0] and math.isclose(g[-1], f[-1] / 32, rel_tol=1e-13) and (np.diff(g) < 0).all()


@pytest.mark.parametrize("args", [(0, 10000.0), (7, 10000.0), (64, 1.0), (64, float("nan"))])
def test_frequencies_refuse(args):
    with pytest.raises(tq.TQError) as e:
        tq.rope_frequencies(*args)
    assert e.value.status == 1


def test_frequencies_refuse_scalings():
    with pytest.raises(ValueError):
        tq.rope_frequencies(64, 10000.0, "cubic")
    for kw in (dict(scaling="linear", factor=0.0), dict(scaling="bands", factor=8.0), dict(scaling="yarn", factor=8.0),
               dict(scaling="bands", factor=8.0, original_len=8192, low=4.0, high=4.0),
               dict(scaling="yarn", factor=8.0, original_len=4096, low=0.0)):
        with pytest.raises(tq.TQError):
            tq.rope_frequencies(64, 10000.0, **kw)


def _call(x=4096, out=4096, heads=2, dtype=0, n=3, D=8, rot=8, freq=4096, pos=4096, bits=32, flags=0, nt=1):
    """A call with made-up addresses: only for arguments that are refused before anything is launched."""
    t = (tq._RopeTensor * 2)()
    for i in range(2):
        t[i] = tq._RopeTensor(x, out, heads, 16, 8, 16, 8)
    return tq.lib().tq_rope(t, nt, dtype, n, D, rot, freq, pos, bits, 1.0, flags, None)


@pytest.mark.parametrize("kw,status", [
    (dict(nt=0), 1), (dict(nt=3), 1), (dict(dtype=3), 1), (dict(n=-1), 1), (dict(D=0), 1), (dict(rot=0), 1),
    (dict(rot=3), 1), (dict(rot=10), 1), (dict(D=8192, rot=8), 2), (dict(bits=16), 1), (dict(flags=4), 1),
    (dict(heads=-1), 1), (dict(x=0), 1), (dict(out=0), 1), (dict(x=4098), 2), (dict(out=4097, dtype=1), 2),
    (dict(freq=0), 1), (dict(pos=0), 1),
])
def test_refusals(kw, status):
    assert _call(**kw) == status
    assert tq.lib().tq_last_error()


def test_no_tokens_is_no_work():
    assert _call(n=0, x=0, out=0, freq=0, pos=0) == 0


# ------------------------------------------------------------------ GPU
def _ref(x, pos, freq, inter, factor=1.0, back=False):
    r = 2 * len(freq)
    a = pos.astype(np.float64)[:, None] * freq
    z = factor * np.exp((-1j if back else 1j) * a)[:, None]
    y = x.astype(np.float64).copy()
    i = np.arange(r // 2)
    u, v = (2 * i, 2 * i + 1) if inter else (i, i + r // 2)
    w = (y[..., u] + 1j * y[..., v]) * z
    size = np.zeros_like(y)
    size[..., u] = size[..., v] = np.abs(x[..., u]) + np.abs(x[..., v])
    y[..., u], y[..., v] = w.real, w.imag
    return y, size * factor


def _check(got, x, pos, freq, inter, factor=1.0, back=False, label=""):
    """The angle is good to pi 2^-24 (rounding of the fraction of a half turn) and its sine and cosine to two units more
    (2^-22 in all, with the factor's rounding); two products and a sum add three roundings of 2^-24."""
    y, size = _ref(x, pos, freq, inter, factor, back)
    g = got.double().cpu().numpy()
    r = 2 * len(freq)
    tol = (math.pi * 2.0 ** -24 + 2.0 ** -22 + 3 * 2.0 ** -24) * size
    tol = tol + torch.finfo(got.dtype).eps / 2 * (np.abs(y) + tol) + (2.0 ** -25 if got.dtype == torch.float16 else 0)
    assert (np.abs(g - y)[..., :r] <= tol[..., :r]).all(), (label, np.abs(g - y).max())
    assert np.array_equal(g[..., r:], x[..., r:].astype(np.float64)), label


def _np(t):
    return t.float().cpu().numpy()


CASES = [  # n, Hq, Hkv, D, rot, dtype, interleaved
    (1, 32, 8, 128, 128, torch.bfloat16, False),
    (64, 32, 8, 128, 128, torch.float16, True),
    (7, 5, 1, 96, 40, torch.float32, True),
    (300, 4, 4, 80, 80, torch.bfloat16, False),      # halves of 40: 8 at a time
    (33, 3, 3, 80, 20, torch.float16, False),        # halves of 10: 2 at a time
    (33, 3, 1, 50, 22, torch.bfloat16, True),        # rest of 28
    (9, 2, 1, 10, 2, torch.float32, False),          # one pair
    (1025, 1, 1, 64, 32, torch.bfloat16, False),     # several tokens a block, a ragged last one
    (2, 64, 64, 256, 256, torch.float32, False),
]


@gpu
@pytest.mark.parametrize("n,Hq,Hkv,D,rot,dtype,inter", CASES)
def test_rope_matches_the_definition(n, Hq, Hkv, D, rot, dtype, inter):
    g = torch.Generator(device=DEV).manual_seed(n + D)
    q, k = (torch.randn(n, h, D, generator=g, device=DEV).to(dtype) for h in (Hq, Hkv))
    pos = torch.randint(0, 131072, (n,), generator=g, device=DEV, dtype=torch.int32)
    freq, _ = tq.rope_frequencies(rot, 10000.0)
    qo, ko = tq.rope(q, k, pos, torch.tensor(freq, device=DEV), interleaved=inter)
    for x, y in ((q, qo), (k, ko)):
        assert y.dtype == dtype and y.shape == x.shape
        _check(y, _np(x), pos.cpu().numpy(), freq, inter, label="forward")
    back, none = tq.rope(q, None, pos, torch.tensor(freq, device=DEV), interleaved=inter, factor=1.25, transpose=True)
    assert none is None
    _check(back, _np(q), pos.cpu().numpy(), freq, inter, 1.25, True, label="transposed")


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shift", [0, 1, 2])
def test_rope_strided_unaligned_and_in_place(dtype, shift):
    """Queries and keys as slices of one projection row, from an odd element on, and written over themselves."""
    n, Hq, Hkv, D = 37, 6, 2, 64
    g = torch.Generator(device=DEV).manual_seed(shift)
    rows = torch.randn(n, (Hq + 2 * Hkv) * D + 3, generator=g, device=DEV).to(dtype)
    before = rows.clone()
    q = rows[:, shift:shift + Hq * D].unflatten(1, (Hq, D))
    k = rows[:, shift + Hq * D:shift + (Hq + Hkv) * D].unflatten(1, (Hkv, D))
    qx, kx = _np(q), _np(k)
    pos = torch.arange(n, device=DEV) * 1000 - 5                      # int64, some negative
    freq, factor = tq.rope_frequencies(48, 10000.0, "yarn", factor=4.0, original_len=4096)
    f = torch.tensor(freq, device=DEV)
    a, b = tq.rope(q, k, pos, f, factor=factor)
    _check(a, qx, pos.cpu().numpy(), freq, False, factor)
    _check(b, kx, pos.cpu().numpy(), freq, False, factor)
    assert torch.equal(rows, before)
    tq.rope(q, k, pos, f, factor=factor, q_out=q, k_out=k)
    assert torch.equal(q, a) and torch.equal(k, b)
    assert torch.equal(rows[:, :shift], before[:, :shift])
    assert torch.equal(rows[:, shift + (Hq + Hkv) * D:], before[:, shift + (Hq + Hkv) * D:])


@gpu
@pytest.mark.parametrize("n,Hq,Hkv,D,rot,dtype,inter", [
    (1, 1, 0, 8, 2, torch.bfloat16, False),          # one row of one piece
    (5, 32, 8, 128, 50, torch.bfloat16, False),
    (2500, 6, 2, 80, 54, torch.float16, True),       # several tokens a block, a ragged last one
    (700, 28, 4, 96, 90, torch.float32, False),
    (3, 200, 56, 256, 250, torch.bfloat16, True),    # a token in several slices
    (2, 3, 1, 4096, 4094, torch.float32, False),     # one row a block
])
def test_rope_narrow_halves_in_whole_rows(n, Hq, Hkv, D, rot, dtype, inter):
    """Halves that are no multiples of 16 bytes in rows that are: against the definition, in place inside a wider row,
    and bit for bit what the same rows give from an address that is not aligned."""
    g = torch.Generator(device=DEV).manual_seed(n + rot)
    q, k = (torch.randn(n, h, D, generator=g, device=DEV).to(dtype) for h in (Hq, Hkv))
    pos = torch.randint(0, 1 << 20, (n,), generator=g, device=DEV)
    freq, _ = tq.rope_frequencies(rot, 10000.0)
    f = torch.tensor(freq, device=DEV)
    qo, ko = tq.rope(q, k, pos, f, interleaved=inter)
    _check(qo, _np(q), pos.cpu().numpy(), freq, inter, label="q")
    _check(ko, _np(k), pos.cpu().numpy(), freq, inter, label="k")
    for shift in (0, 1):
        wide = torch.full((n, 16 + (Hq + Hkv) * D + 16), 7.0, device=DEV, dtype=dtype)
        a = wide[:, 16 - shift:16 - shift + Hq * D].unflatten(1, (Hq, D))
        b = wide[:, 16 - shift + Hq * D:16 - shift + (Hq + Hkv) * D].unflatten(1, (Hkv, D))
        a.copy_(q)
        b.copy_(k)
        tq.rope(a, b, pos, f, interleaved=inter, q_out=a, k_out=b)
        assert torch.equal(a, qo) and torch.equal(b, ko), shift
        assert (wide[:, :16 - shift] == 7).all() and (wide[:, 16 - shift + (Hq + Hkv) * D:] == 7).all()


@gpu
def test_rope_far_positions():
    """Positions up to 2^31 in 32 bits and 2^40 in 64: the angle keeps 64-bit turns.  The product pos * freq / 2 pi is
    rounded twice (2^-52 relative), which at 2^40 turns / 2 pi is 2 pi 2^-14.6 of an angle; at 2^31 2 pi 2^-23.6."""
    freq = np.array([1.0, 0.37, 1e-3, 1e-6])
    x = torch.randn(4, 1, 8, device=DEV, generator=torch.Generator(device=DEV).manual_seed(0))
    for pos, err in ((torch.tensor([2 ** 31 - 1, -2 ** 31, 12345678, 3], dtype=torch.int32, device=DEV), 2.0 ** -52),
                     (torch.tensor([2 ** 40, 2 ** 40 - 1, -2 ** 39, 2 ** 33 + 7], device=DEV), 2.0 ** -52)):
        got, _ = tq.rope(x, None, pos, torch.tensor(freq, device=DEV))
        y, size = _ref(_np(x), pos.cpu().numpy(), freq, False)
        a = np.abs(pos.cpu().numpy().astype(np.float64))[:, None] * freq
        angle = np.concatenate([a, a], 1)[:, None] * err * 2              # the reference's own product is rounded too
        tol = (angle + math.pi * 2.0 ** -24 + 2.0 ** -22 + 4 * 2.0 ** -24) * size
        assert (np.abs(got.double().cpu().numpy() - y) <= tol).all()


@gpu
def test_rope_gradient_is_the_transposed_rotation():
    """<g, rope(x)> is linear in x: its differences are its gradient, rope(g, transpose=True).  Both sides are sums of
    128 terms of 32-bit results good to 5e-7 of |g| |x|."""
    gen = torch.Generator(device=DEV).manual_seed(3)
    x, g, d = (torch.randn(5, 2, 128, generator=gen, device=DEV) for _ in range(3))
    pos = torch.randint(0, 9999, (5,), generator=gen, device=DEV)
    freq, _ = tq.rope_frequencies(96, 10000.0)
    f = torch.tensor(freq, device=DEV)
    grad, _ = tq.rope(g, None, pos, f, factor=1.5, transpose=True)
    up, _ = tq.rope(x + d, None, pos, f, factor=1.5)
    dn, _ = tq.rope(x - d, None, pos, f, factor=1.5)
    left = ((up.double() - dn.double()) * g.double()).sum(-1) / 2
    right = (grad.double() * d.double()).sum(-1)
    size = (g.double().abs() * (x.double().abs() + d.double().abs() + 1)).sum(-1)
    assert ((left - right).abs() <= 4 * 5e-7 * 1.5 * size).all()
    y = x.double().requires_grad_()
    a = pos.double()[:, None, None] * f
    u, v, rest = y[..., :48], y[..., 48:96], y[..., 96:]
    out = torch.cat([1.5 * (u * a.cos() - v * a.sin()), 1.5 * (v * a.cos() + u * a.sin()), rest], -1)
    out.backward(g.double())
    assert ((grad.double() - y.grad).abs() <= 1e-6 * 1.5 * (g.abs().amax())).all()


@gpu
def test_rope_streams_graphs_and_edges():
    freq, _ = tq.rope_frequencies(128, 10000.0)
    f = torch.tensor(freq, device=DEV)
    q = torch.randn(5, 4, 128, device=DEV).bfloat16()
    pos = torch.arange(5, device=DEV, dtype=torch.int32)
    want, _ = tq.rope(q, None, pos, f)
    out = torch.empty_like(q)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    tq.rope(q, None, pos, f, q_out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tq.rope(q, None, pos, f, q_out=out)
    pos += 7
    graph.replay()
    again, _ = tq.rope(q, None, pos, f)
    assert torch.equal(out, again) and not torch.equal(again, want)
    empty, k = tq.rope(q[:0], q[:0, :1], pos[:0], f)
    assert empty.shape == (0, 4, 128) and k.shape == (0, 1, 128)
    none, k = tq.rope(q[:, :0], q, pos, f)
    assert none.shape == (5, 0, 128) and torch.equal(k, again)


@gpu
def test_rope_refuses_tensors():
    f = torch.ones(4, dtype=torch.float64, device=DEV)
    q = torch.zeros(3, 2, 8, device=DEV)
    pos = torch.zeros(3, dtype=torch.int32, device=DEV)
    for bad in (lambda: tq.rope(q.cpu(), None, pos, f), lambda: tq.rope(q, None, pos.cpu(), f),
                lambda: tq.rope(q, None, pos, f.float()), lambda: tq.rope(q, None, pos[:2], f),
                lambda: tq.rope(q, q.half(), pos, f), lambda: tq.rope(q, None, pos.float(), f),
                lambda: tq.rope(q.transpose(1, 2), None, pos, f), lambda: tq.rope(q, None, pos, f, q_out=q[:2])):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(tq.TQError):
        tq.rope(q, None, pos, torch.ones(5, dtype=torch.float64, device=DEV))    # rot 10 > D
    with pytest.raises(TypeError):
        tq.rope(q.double(), None, pos, f)

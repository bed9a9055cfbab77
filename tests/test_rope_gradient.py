"""Gradients of tq.rope through autograd."""
import numpy as np
import pytest

import kv_cache_vector_08_b200 as tq

torch = pytest.importorskip("torch")
gpu = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def _plain(x, pos, f, inter, factor):
    """The rotation in 64 bits, by elementary operations that autograd follows."""
    r = 2 * f.shape[0]
    a = pos.double()[:, None, None] * f
    u, v = (x[..., 0:r:2], x[..., 1:r:2]) if inter else (x[..., :r // 2], x[..., r // 2:r])
    y, z = factor * (u * a.cos() - v * a.sin()), factor * (v * a.cos() + u * a.sin())
    turned = torch.stack([y, z], -1).flatten(-2) if inter else torch.cat([y, z], -1)
    return torch.cat([turned, x[..., r:]], -1)


def _data(n, Hq, Hkv, D, rot, dtype, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    q, k, gq, gk = (torch.randn(n, h, D, generator=g, device=DEV).to(dtype) for h in (Hq, Hkv, Hq, Hkv))
    pos = torch.randint(0, 9999, (n,), generator=g, device=DEV)
    f = torch.tensor(tq.rope_frequencies(rot, 10000.0)[0], device=DEV)
    return q, k, gq, gk, pos, f


@gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("inter,transpose,rot", [(False, False, 96), (True, False, 128), (False, True, 50), (True, True, 2)])
def test_gradients_match_the_formula(dtype, inter, transpose, rot):
    """Against autograd in 64 bits.  A gradient is turned as the values are: angles of up to 9,999 are good to pi 2^-24
    and their sines to 2^-22 with the factor, two products and a sum add 3 2^-24, each relative to the two elements of
    the pair; then half a step of the type."""
    q, k, gq, gk, pos, f = _data(7, 4, 2, 128, rot, dtype)
    qs, ks = q.clone().requires_grad_(), k.clone().requires_grad_()
    outs = tq.rope(qs, ks, pos, f, interleaved=inter, factor=1.25, transpose=transpose)
    with torch.no_grad():
        same = tq.rope(qs, ks, pos, f, interleaved=inter, factor=1.25, transpose=transpose)
    assert all(torch.equal(a, b) and a.requires_grad and not b.requires_grad for a, b in zip(outs, same))
    torch.autograd.backward(outs, (gq, gk))
    for x, got, g in ((q, qs.grad, gq), (k, ks.grad, gk)):
        x = x.double().requires_grad_()
        _plain(x, -pos if transpose else pos, f, inter, 1.25).backward(g.double())
        size = 1.25 * 2 * g.double().abs().amax(-1, keepdim=True)
        tol = (np.pi * 2.0 ** -24 + 2.0 ** -22 + 3 * 2.0 ** -24) * size
        tol = tol + torch.finfo(dtype).eps / 2 * (x.grad.abs() + tol) + (2.0 ** -25 if dtype == torch.float16 else 0)
        assert got.dtype == dtype and ((got.double() - x.grad).abs() <= tol).all()


@gpu
def test_gradients_match_differences():
    """The sum of g rope(x) is linear in x, so a central difference of any width is its derivative; both sides are sums
    of 2 x 128 products of values good to 5e-7 relative to |g| |x|."""
    q, k, gq, gk, pos, f = _data(5, 2, 1, 128, 96, torch.float32, 1)
    d = torch.randn_like(q)
    x = q.clone().requires_grad_()
    (tq.rope(x, None, pos, f, factor=1.5)[0] * gq).sum().backward()
    up, dn = (tq.rope(q + s * d, None, pos, f, factor=1.5)[0].double() for s in (1, -1))
    left, right = ((up - dn) / 2 * gq.double()).sum(-1), (x.grad.double() * d.double()).sum(-1)
    size = (gq.double().abs() * (q.double().abs() + d.double().abs() + 1)).sum(-1)
    assert ((left - right).abs() <= 4 * 5e-7 * 1.5 * size).all()


@gpu
def test_only_what_is_asked_for_gets_a_gradient():
    q, k, gq, gk, pos, f = _data(6, 3, 2, 64, 64, torch.float32, 2)
    ks = k.clone().requires_grad_()
    a, b = tq.rope(q, ks, pos, f)
    assert not a.requires_grad and b.requires_grad
    b.backward(gk)
    assert q.grad is None and torch.equal(ks.grad, tq.rope(gk, None, pos, f, transpose=True)[0])
    qs, ks = q.clone().requires_grad_(), k.clone().requires_grad_()
    tq.rope(qs, ks, pos, f)[1].sum().backward()                    # an expanded gradient, and none for q
    assert qs.grad is None and torch.equal(ks.grad, tq.rope(torch.ones_like(k), None, pos, f, transpose=True)[0])
    wide = torch.randn(6, 3, 256, device=DEV, requires_grad=True)  # a slice of wider rows, its gradient every other channel
    y = tq.rope(wide[..., :64], None, pos, f)[0]
    y.backward(torch.stack([gq, gq], -1)[..., 0])
    assert torch.equal(wide.grad[..., :64], tq.rope(gq, None, pos, f, transpose=True)[0]) and (wide.grad[..., 64:] == 0).all()
    x = torch.zeros(0, 3, 64, device=DEV, requires_grad=True)
    tq.rope(x, None, pos[:0], f)[0].sum().backward()
    assert x.grad.shape == x.shape


@gpu
def test_a_gradient_has_a_gradient():
    q, _, gq, gk, pos, f = _data(4, 2, 1, 64, 32, torch.float32, 3)
    x, g = q.clone().requires_grad_(), gq.clone().requires_grad_()
    y = tq.rope(x, None, pos, f, interleaved=True)[0]
    (dx,) = torch.autograd.grad(y, x, g, create_graph=True)
    (dg,) = torch.autograd.grad(dx, g, q)                          # <dx, q> = <g, rope(q)>
    assert torch.equal(dg, tq.rope(q, None, pos, f, interleaved=True)[0])


@gpu
def test_a_gradient_on_a_given_stream():
    """Forward on the given stream, backward on it too: autograd orders it behind the current one."""
    q, k, gq, gk, pos, f = _data(513, 8, 2, 128, 128, torch.bfloat16, 4)
    want = [tq.rope(g, None, pos, f, transpose=True)[0] for g in (gq, gk)]
    side = torch.cuda.Stream()
    for _ in range(5):
        side.wait_stream(torch.cuda.current_stream())
        qs, ks = q.clone().requires_grad_(), k.clone().requires_grad_()
        side.wait_stream(torch.cuda.current_stream())
        a, b = tq.rope(qs, ks, pos, f, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        torch.autograd.backward((a, b), (gq, gk))
        assert torch.equal(qs.grad, want[0]) and torch.equal(ks.grad, want[1])


@gpu
def test_what_cannot_have_a_gradient_is_refused():
    q, k, gq, gk, pos, f = _data(3, 2, 1, 64, 64, torch.float32, 5)
    x = q.clone().requires_grad_()
    for bad in (lambda: tq.rope(x, None, pos, f, q_out=torch.empty_like(q)), lambda: tq.rope(q, x, pos, f, k_out=q.clone()),
                lambda: tq.rope(q, None, pos, f.clone().requires_grad_())):
        with pytest.raises(ValueError):
            bad()
    with torch.no_grad():
        out = torch.empty_like(q)
        tq.rope(x, None, pos, f.clone().requires_grad_(), q_out=out)
        assert torch.equal(out, tq.rope(q, None, pos, f)[0])
        leaf = q.clone().requires_grad_()
        tq.rope(leaf, None, pos, f, q_out=leaf)                    # in place, as any operation under no_grad
        assert torch.equal(leaf, out)

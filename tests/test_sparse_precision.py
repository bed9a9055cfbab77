"""tq_sparse_decode_attention and tq_decode_attention against the definition in 64 bits, to the precision of the decode
kernel's own arithmetic (which is well above that of fp16 operands)."""
import math

import numpy as np
import pytest

import cacheref
import kv_cache_vector_08_b200 as tq

torch = pytest.importorskip("torch")
gpu = pytest.mark.gpu
DEV = torch.device("cuda", 0)
D = 128
FIX = 32000.0            # steps of the fixed-point queries and key levels over their largest value


def _attend(cache, b, h, q, tokens, scale):
    """q [R, D] over `tokens` -> (out, tolerance).

    The kernel carries a key level in steps of max|c| / 32000 and the coordinates of Pi q and S q in steps of their
    largest / 32000; a value so rounded is off by step / sqrt(12) in the mean square.  The logit of token t is then off by
      d_t = scale n_t sqrt( |Pi q|^2 step_c^2 + |c_t|^2 step_q^2 + (sqrt(pi/2)/w r_t)^2 w step_s^2 ) / sqrt(12)
    over the groups, which is the relative error of the weight p_t and moves output channel j by p_t d_t (v_tj - o_j).
    A value level is rounded once to fp16, by e(c) that the codebook gives; the rotated coordinate i is off by
    sum_t p_t n_t e(c_ti), which the rotation spreads evenly over its channels.  These are sums of independent terms, of
    which six standard deviations are allowed.  Exponentials, sums and weights (two fp16 parts) are good to 2^-20 of the
    root of the sum of the squares of what they add, or of a weight's own size for all."""
    s = cache.slots(b, h, tokens)
    R, L = len(q), len(tokens)
    logit, dvar = np.zeros((R, L)), np.zeros((R, L))
    v, off = np.zeros((L, D)), np.zeros((L, D))
    for g, (w, kb, vb) in enumerate(cache.groups):
        sl = slice(cache.off[g], cache.off[g + 1])
        x, kc, p = q[:, sl], cache.k[g], cache.kp[g]
        n, r = kc["norm"][s].astype(np.float64), kc["rnorm"][s].astype(np.float64)
        pq, sq, c = x @ p["Pi"].T, x @ p["S"].T, p["centroids"][kc["idx"][s]]
        f = math.sqrt(math.pi / 2) / w * r
        logit += n * (pq @ c.T + f * (sq @ (2.0 * kc["signs"][s] - 1).T))
        step_q, step_s = np.abs(pq).max(1) / FIX, np.abs(sq).max(1) / FIX
        step_c = np.abs(p["centroids"]).max() / FIX
        dvar += n ** 2 / 12 * (((pq ** 2).sum(1) * step_c ** 2)[:, None] + step_q[:, None] ** 2 * (c ** 2).sum(1)
                               + step_s[:, None] ** 2 * f ** 2 * w)
        vc, p = cache.v[g], cache.vp[g]
        vn, level = vc["norm"][s].astype(np.float64)[:, None], p["centroids"]
        half = level.astype(np.float32).astype(np.float16).astype(np.float64)
        v[:, sl] = (vn * level[vc["idx"][s]]) @ p["Pi"]
        off[:, sl] = np.sqrt(((vn * (half - level)[vc["idx"][s]]) ** 2).sum(1, keepdims=True) / w)
    logit, d2 = logit * scale, dvar * scale ** 2
    p = np.exp(logit - logit.max(1, keepdims=True))
    p /= p.sum(1, keepdims=True)
    out = p @ v
    w2 = p ** 2 * d2
    moved = np.maximum(w2 @ v ** 2 - 2 * out * (w2 @ v) + out ** 2 * w2.sum(1)[:, None], 0)
    small = 2.0 ** -20 * (np.sqrt(p ** 2 @ v ** 2) + np.abs(out) + np.sqrt((out ** 2).mean(1, keepdims=True)))
    return out, 6 * (np.sqrt(moved) + np.sqrt(p ** 2 @ off ** 2)) + 6 * small


@gpu
@pytest.mark.parametrize("kind", sorted(cacheref.LAYOUTS))
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("qscale,spread,size", [(1.0, 0.5, 1.0), (8.0, 0.5, 1.0), (0.1, 0.0, 1e-2)])
def test_sparse_keeps_the_precision_of_the_decode_kernel(kind, dtype, qscale, spread, size):
    """Ordinary, peaked and flat weights, the last over values around 0.01."""
    rng = np.random.default_rng(11)
    B, Hq, Hkv, page, select, lens = 2, 8, 2, 64, 6, [64 * 20 - 9, 64 * 7]
    max_len, rep, scale = 64 * 20, Hq // Hkv, 1 / math.sqrt(D)
    cache = cacheref.Cache(rng, kind, B, Hkv, lens, max_len, page, spread=spread)
    for (w, _, _), vc in zip(cache.groups, cache.v):
        vc["norm"] = (vc["norm"].astype(np.float64) * size).astype(np.float16)
    kc, vc, table = cacheref.upload(cache, DEV)
    kctx, vctx = cacheref.contexts(kind)
    q = torch.tensor(qscale * rng.standard_normal((B, Hq, D)), device=DEV).to(dtype)
    box = torch.randn(cache.pool, Hkv, 2, D, device=DEV, generator=torch.Generator(device=DEV).manual_seed(1)).sort(2).values
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    out, sel = tq.sparse_decode_attention(kctx, vctx, cache.off, q, box, kc, vc, sl, Hkv, max_len, scale, block_table=table,
                                          page_tokens=page, select=select)
    full = None
    if dtype != torch.float16:
        full = tq.decode_attention(kctx, vctx, cache.off, q, kc, vc, sl, Hkv, max_len, scale, block_table=table, page_tokens=page)
    assert kctx[0].device_error() == 0
    qn, sel = q.double().cpu().numpy(), sel.cpu().numpy()
    for b in range(B):
        for h in range(Hkv):
            rows = slice(h * rep, (h + 1) * rep)
            t = (sel[b, h][sel[b, h] >= 0][:, None] * page + np.arange(page)).reshape(-1)
            ref, tol = _attend(cache, b, h, qn[b, rows], t[t < lens[b]], scale)
            cacheref.check(out[b, rows], ref, tol, dtype, "sparse")
            if full is not None:
                ref, tol = _attend(cache, b, h, qn[b, rows], np.arange(lens[b]), scale)
                cacheref.check(full[b, rows], ref, tol, torch.float32, "decode")

"""tq_tree_attention: values far below 1, whose weighted means fall into fp16's fixed steps unless a row is scaled."""
import math

import numpy as np
import pytest

import cacheref
import kv_cache_vector_08_b200 as tq

torch = pytest.importorskip("torch")
gpu = pytest.mark.gpu
DEV = torch.device("cuda", 0)
D = 128


@gpu
@pytest.mark.parametrize("size", [1.0, 1e-1, 1e-2, 1e-3])
@pytest.mark.parametrize("kind,Hq,Hkv,T,lens", [
    ("4", 8, 2, 3, [4000]),                    # 12 rows, four copies of each; many splits
    ("2.5", 8, 2, 10, [3000]),                 # 40 rows, two copies
    ("3.5", 8, 1, 20, [2500, 40]),             # 160 rows, two row tiles
    ("3", 160, 160, 2, [200]),                 # more blocks than SMs: one split, written without a merge
])
def test_small_values_keep_the_precision_of_large_ones(kind, Hq, Hkv, T, lens, size):
    """All value norms around `size`, weights nearly flat over thousands of tokens.

    cacheref.attend's tolerance is relative to the values but for a floor of 1e-6, which is taken off here.  Below norms
    of about 1 a second kind of rounding joins those it counts: an element of V under 2^-14 is rounded to a multiple of
    2^-24, by 2^-25 at most and 2^-25 / sqrt(3) in the mean square.  At a norm of 1e-3 an element is 1e-3 / sqrt(128) =
    8.8e-5 in the mean square, so that is 2e-4 of it, which with the relative rounding of 2e-4 makes 2.8e-4: within the
    4e-4 that the tolerance has for them.  Of a row as a whole: weights and output and last rotation 2e-4 each, values
    2.8e-4, logits next to nothing (they hardly differ), in all 4.5e-4; twice that is allowed."""
    rng = np.random.default_rng(len(lens) + T)
    B, max_len, scale = len(lens), max(lens), 0.1 / math.sqrt(D)
    cache = cacheref.Cache(rng, kind, B, Hkv, lens, max_len)
    for (w, _, _), v in zip(cache.groups, cache.v):
        v["norm"] = (v["norm"].astype(np.float64) * (size / math.sqrt(w))).astype(np.float16)
    kc, vc, _ = cacheref.upload(cache, DEV)
    kctx, vctx = cacheref.contexts(kind)
    q = rng.standard_normal((B, T, Hq, D)).astype(np.float32)
    out = tq.tree_attention(kctx, vctx, cache.off, torch.tensor(q, device=DEV), kc, vc,
                            torch.tensor(lens, dtype=torch.int32, device=DEV), Hkv, max_len, scale)
    torch.cuda.synchronize()
    assert kctx[0].device_error() == 0
    rep = Hq // Hkv
    for b in range(B):
        keep = np.ones((T, lens[b]), bool)
        keep[:, lens[b] - T:] = np.tril(np.ones((T, T), bool))
        for h in range(0, Hkv, max(1, Hkv // 16)):
            rows = q[b, :, h * rep:(h + 1) * rep].reshape(T * rep, D).astype(np.float64)
            ref, tol = cache.attend(b, h, rows, np.arange(lens[b]), np.repeat(keep, rep, 0), scale)
            got = out[b, :, h * rep:(h + 1) * rep].reshape(T * rep, D)
            cacheref.check(got, ref, tol - 1e-6, torch.float32, "values of %g" % size)
            off = np.linalg.norm(got.double().cpu().numpy() - ref, axis=1) / np.linalg.norm(ref, axis=1)
            assert off.max() <= 9e-4, (b, h, off.max())

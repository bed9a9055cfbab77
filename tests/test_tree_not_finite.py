"""tq_tree_attention: a norm that is not finite makes every output of the rows that attend its token NaN, and no other."""
import math

import numpy as np
import pytest

import cacheref
import kv_cache_vector_08_b200 as tq

torch = pytest.importorskip("torch")
gpu = pytest.mark.gpu
DEV = torch.device("cuda", 0)
D, T = 128, 6


def _run(cache, kind, q, length, mask):
    kc, vc, _ = cacheref.upload(cache, DEV)
    kctx, vctx = cacheref.contexts(kind)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    out = tq.tree_attention(kctx, vctx, cache.off, q, kc, vc, i32(length), cache.Hkv, cache.max_len, 1 / math.sqrt(D), i32(T),
                            torch.tensor(mask, device=DEV))
    torch.cuda.synchronize()
    assert kctx[0].device_error() == 0
    return out


@gpu
@pytest.mark.parametrize("kind,groups", [("4", [0]), ("2.5", [0, 1]), ("3.5", [1])])
@pytest.mark.parametrize("which", ["key", "residual", "value"])
@pytest.mark.parametrize("value", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("context", [0, 100, 4096])
def test_every_output_of_the_rows_that_attend_it(kind, groups, which, value, context):
    """Drafted tokens 1 and 4.  Row 1 attends the context and token 1 alone, row 4 tokens 0 and 4, row 5 both bad ones;
    row 3 nothing but the context.  With 4,096 tokens of context every tile is a split of its own and the drafts are the
    last: there row 1 has a sum that is NaN and no maximum, row 3 neither."""
    rng = np.random.default_rng(context + len(kind))
    Hq, Hkv, n = 8, 2, context + T
    cache = cacheref.Cache(rng, kind, 1, Hkv, [n], n)
    q = torch.tensor(rng.standard_normal((1, T, Hq, D)), device=DEV).float()
    mask = np.array([0b1, 0b10, 0b101, 0, 0b10001, 0b110010], dtype=np.int64).reshape(1, T, 1)
    assert (tq.tree_workspace_size(1, T, Hq, Hkv, D, len(cache.groups), n) > 256) == (context > 100)   # splits
    want = _run(cache, kind, q, n, mask)
    assert want.isfinite().all()
    store = {"key": [c["norm"] for c in cache.k], "residual": [c["rnorm"] for c in cache.k],
             "value": [c["norm"] for c in cache.v]}[which]
    for g in groups:
        for h in range(Hkv):
            store[g][cache.slots(0, h, np.array([context + 1, context + 4]))] = value
    got = _run(cache, kind, q, n, mask)
    assert torch.equal(got[0, [0, 2, 3]], want[0, [0, 2, 3]])
    assert got[0, [1, 4, 5]].isnan().all()
    if context:
        store[groups[0]][cache.slots(0, 0, np.array([context // 2]))] = value       # a token of the context: every row
        got = _run(cache, kind, q, n, mask)
        rep = Hq // Hkv
        assert got[0, :, :rep].isnan().all() and torch.equal(got[0, [0, 2, 3], rep:], want[0, [0, 2, 3], rep:])

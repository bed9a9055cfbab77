"""Channels of a page in which every key is NaN: from tq_page_bounds through the selection."""
import numpy as np
import pytest

import cacheref
import kv_cache_vector_08_b200 as tq

torch = pytest.importorskip("torch")
gpu = pytest.mark.gpu
DEV = torch.device("cuda", 0)
D = 128


def _score(q, box):
    """[pages] scores of one kv head in 64 bits: q [rep, D], box [pages, 2, D]; a product with a sum of 0 is 0."""
    up, dn = np.maximum(q, 0).sum(0), np.minimum(q, 0).sum(0)
    with np.errstate(invalid="ignore"):
        return np.where(up != 0, up * box[:, 1], 0).sum(1) + np.where(dn != 0, dn * box[:, 0], 0).sum(1)


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("signs", ["positive", "negative", "both", "none"])
def test_a_channel_without_keys_puts_its_page_last(dtype, signs):
    """Pages 2 and 7 hold the largest keys, but all keys of page 2 are NaN in channel 9, and those of page 7 but one.
    Page 2 is bounded by no key there and is taken after all others; page 7 by its one key.  A query of 0 in the channel
    asks nothing of it."""
    rng = np.random.default_rng(3)
    page, pages, Hq, Hkv = 64, 10, 4, 1
    n = page * pages
    cache = cacheref.Cache(rng, "4", 1, Hkv, [n], n, page)
    kc, vc, table = cacheref.upload(cache, DEV)
    kctx, vctx = cacheref.contexts("4")
    k = rng.standard_normal((n, Hkv, D))
    for p in (2, 7):
        k[p * page:(p + 1) * page] *= 8
        k[p * page:(p + 1) * page, :, 9] = np.nan
    k[7 * page + 5, :, 9] = 0.5
    k = torch.tensor(k, device=DEV).to(dtype)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    bounds = tq.page_bounds(k, i32(0, n), i32(0), table, page, tq.alloc_page_bounds(cache.pool, Hkv, D, dtype), n)
    box = bounds.double().cpu().numpy()[cache.table[0]][:, 0]
    assert box[2, 0, 9] == np.inf and box[2, 1, 9] == -np.inf and (box[7, :, 9] == 0.5).all()
    q = rng.standard_normal((1, Hq, D))
    q[0, :, 9] = {"positive": 1.0, "negative": -1.0, "both": [1, -1, 2, -0.5], "none": 0.0}[signs]
    q = torch.tensor(q, device=DEV).to(dtype)
    score = _score(q[0].double().cpu().numpy(), box)
    order = np.argsort(-score, kind="stable")
    assert (order[-1] == 2) == (signs != "none") and (order[0] == 7 or signs == "none")
    for select in (1, 4, 9, 10):
        _, sel = tq.sparse_decode_attention(kctx, vctx, cache.off, q, bounds, kc, vc, i32(n), Hkv, n, 0.1, block_table=table,
                                            page_tokens=page, select=select, first=0, last=0)
        assert sel[0, 0].tolist() == sorted(order[:select].tolist()), select
        _, sel = tq.sparse_decode_attention(kctx, vctx, cache.off, q, bounds, kc, vc, i32(n), Hkv, n, 0.1, block_table=table,
                                            page_tokens=page, select=select, first=3, last=0)
        assert 2 in sel[0, 0].tolist() or select < 3           # in any case among the first

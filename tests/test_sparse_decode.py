"""tq_page_bounds and tq_sparse_decode_attention: page bounds, the selection and the attention over it."""
import ctypes
import math

import numpy as np
import pytest

import cacheref
import kv_cache_vector_08_b200 as tq

torch = pytest.importorskip("torch")
gpu = pytest.mark.gpu
DEV = torch.device("cuda", 0)
D = 128


# ------------------------------------------------------------------ refusals (no GPU: nothing is launched)
def _bounds(k=4096, n=1, dtype=0, cu=4096, start=4096, B=1, Hkv=1, D=8, new=1, table=4096, page=64, pages=1, out=4096, np_=1):
    return tq.lib().tq_page_bounds(k, n, dtype, 8, 8, cu, start, B, Hkv, D, new, table, page, pages, out, np_, None)


@pytest.mark.parametrize("kw,status", [
    (dict(dtype=5), 1), (dict(n=-1), 1), (dict(B=-1), 1), (dict(Hkv=0), 1), (dict(D=0), 1), (dict(new=-1), 1), (dict(page=0), 1),
    (dict(pages=-1), 1), (dict(np_=-1), 1), (dict(D=264), 2), (dict(B=65536), 2), (dict(Hkv=65536), 2), (dict(k=0), 1),
    (dict(cu=0), 1), (dict(start=0), 1), (dict(table=0), 1), (dict(out=0), 1), (dict(k=4097, dtype=1), 2),
    (dict(out=4098), 2),
])
def test_bounds_refusals(kw, status):
    assert _bounds(**kw) == status


def test_bounds_without_work():
    assert _bounds(n=0, k=0) == 0 and _bounds(B=0, k=0) == 0 and _bounds(new=0, k=0) == 0 and _bounds(pages=0, k=0) == 0 and _bounds(np_=0, k=0) == 0


def _sparse(select=4, first=1, last=1, page=64, table=4096, bounds=4096, bdtype=1, bpages=4, max_len=256, opts=True):
    o = tq._SparseOpts(bounds, bdtype, bpages, select, first, last, None, table, page, None)
    return tq.lib().tq_sparse_decode_attention(None, None, None, 1, None, 1, None, None, None, 1, 8, 2, 128, max_len, 1.0,
                                               None, ctypes.byref(o) if opts else None, None, 0, None)


@pytest.mark.parametrize("kw", [
    dict(opts=False), dict(select=0), dict(first=-1), dict(last=-1), dict(page=0), dict(page=96), dict(page=128, max_len=192),
    dict(table=None), dict(bounds=None), dict(bdtype=7), dict(bpages=-1), dict(),          # (the last: NULL contexts)
])
def test_sparse_refusals(kw):
    assert _sparse(**kw) == 1


def test_sparse_workspace_size():
    assert tq.sparse_workspace_size(2, 8, 3, D, 1, 256, 64, 4) == 0      # Hq not a multiple of Hkv
    assert tq.sparse_workspace_size(2, 8, 2, D, 1, 256, 64, 0) == 0
    assert 0 < tq.sparse_workspace_size(2, 8, 2, D, 1, 256, 64, 4) < tq.sparse_workspace_size(2, 8, 2, D, 1, 65536, 64, 4)


# ------------------------------------------------------------------ bounds
def _bounds_ref(bounds, k, cu, start, table, page):
    out = bounds.copy()
    pages = out.shape[0]
    for b in range(len(start)):
        for i in range(cu[b + 1] - cu[b]):
            t = start[b] + i
            if t // page >= table.shape[1] or not 0 <= table[b, t // page] < pages:
                continue
            box = out[table[b, t // page]]
            if t % page == 0:
                box[:, 0], box[:, 1] = np.inf, -np.inf
            box[:, 0] = np.fmin(box[:, 0], k[cu[b] + i])
            box[:, 1] = np.fmax(box[:, 1], k[cu[b] + i])
    return out


@gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("Hkv,width,page,new,start", [
    (8, 128, 64, [1, 1, 1], [0, 63, 64]),             # single tokens: a page's first, its last, the next one's first
    (2, 128, 64, [130, 0, 5], [0, 10, 60]),           # whole pages, nothing, across a border
    (1, 64, 128, [300], [17]),
    (3, 100, 64, [65, 64], [1, 64]),                  # 100 channels: 4-byte vectors of no use, one element at a time
    (2, 256, 256, [513], [0]),
])
def test_bounds_match(dtype, Hkv, width, page, new, start):
    rng = np.random.default_rng(len(new) * width)
    B, per = len(new), 10
    pool = B * per + 3
    table = rng.permutation(pool)[:B * per].astype(np.int32).reshape(B, per)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    rows = torch.randn(int(cu[-1]) + 2, 2 * Hkv, width, device=DEV).to(dtype)
    k = rows[:, Hkv:]                                                   # a slice of wider rows
    rows[0, Hkv, 3] = float("nan")                                      # skipped
    rows[1:2, Hkv + Hkv - 1, 5] = float("inf")
    bounds = torch.randn(pool, Hkv, 2, width, device=DEV).to(dtype)
    dev = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    want = _bounds_ref(bounds.float().cpu().numpy(), k.float().cpu().numpy(), cu, start, table, page)
    got = tq.page_bounds(k[:int(cu[-1])], dev(cu), dev(start), dev(table), page, bounds, max(new))
    assert got is bounds
    assert np.array_equal(got.float().cpu().numpy(), want)
    small = torch.randn(pool, Hkv, 2, width, device=DEV).to(dtype)
    want = _bounds_ref(small.float().cpu().numpy(), k.float().cpu().numpy(), cu, start, table, page)
    tq.page_bounds(k[:int(cu[-1])], dev(cu), dev(start), dev(table), page, small, 1)     # more new rows than announced
    assert np.array_equal(small.float().cpu().numpy(), want)


@gpu
def test_bounds_token_by_token_and_bad_pages():
    """Appending one token at a time gives the bounds of all at once; tokens past the table or in pages outside the
    pool leave everything as it was."""
    page, n = 64, 150
    k = torch.randn(n, 2, D, device=DEV).bfloat16()
    table = torch.tensor([[2, 0, 1]], dtype=torch.int32, device=DEV)
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    one, all_ = tq.alloc_page_bounds(3, 2, D, torch.bfloat16), tq.alloc_page_bounds(3, 2, D, torch.bfloat16)
    for t in range(n):
        tq.page_bounds(k[t:t + 1], i(0, 1), i(t), table, page, one, 1)
    tq.page_bounds(k, i(0, n), i(0), table, page, all_, n)
    assert torch.equal(one, all_)
    before = all_.clone()
    for bad in (i(0, -1, 3)[None], i(1, 7, 1 << 30)[None]):
        want = before.float().cpu().numpy()
        want = _bounds_ref(want, k.float().cpu().numpy(), [0, n], [64], np.array([[9, *bad[0, 1:].tolist()]]), page)
        tq.page_bounds(k, i(0, n), i(64), bad.contiguous(), page, all_, n)
        assert np.array_equal(all_.float().cpu().numpy(), want)
    tq.page_bounds(k, i(0, n), i(192), table, page, all_, n)           # past the table
    tq.page_bounds(k, i(5, 5), i(0), table, page, all_, n)             # no rows
    tq.page_bounds(k, i(0, n), i(-4), table, page, all_, n)            # no such token
    tq.page_bounds(k[:n - 1], i(0, n), i(0), table, page, all_, n)     # rows that k does not have
    tq.page_bounds(k, i(-1, 5), i(0), table, page, all_, n)
    assert torch.equal(all_, before)
    with pytest.raises(ValueError):
        tq.page_bounds(k.half(), i(0, n), i(0), table, page, all_, n)
    with pytest.raises(ValueError):
        tq.page_bounds(k, i(0, n).long(), i(0), table, page, all_, n)


# ------------------------------------------------------------------ selection and attention
def _pick(q, box, n, select, first, last):
    """Logical pages of one kv head: q [rep, D], box [pages, 2, D] of its live pages, in 64 bits."""
    with np.errstate(invalid="ignore"):
        s = np.maximum(q[:, None] * box[None, :, 0], q[:, None] * box[None, :, 1]).sum((0, 2))
    s = np.where(np.isnan(s), -np.inf, s)
    p = np.arange(n)
    s[(p < first) | (p >= n - last)] = np.inf
    return np.sort(np.argsort(-s, kind="stable")[:select])


def _case(seed, kind, B, Hq, Hkv, lens, page, select, first, last, dtype, perm=None, box=None):
    rng = np.random.default_rng(seed)
    max_len = max(1, -(-max(lens) // page)) * page
    cache = cacheref.Cache(rng, kind, B, Hkv, lens, max_len, page)
    kc, vc, table = cacheref.upload(cache, DEV)
    q = torch.tensor(rng.standard_normal((B, Hq, D)), device=DEV).to(dtype)
    if box is None:
        mid, half = rng.standard_normal((cache.pool, Hkv, 1, D)), 1 + rng.random((cache.pool, Hkv, 1, D))
        box = torch.tensor(np.concatenate([mid - half, mid + half], 2), device=DEV).to(dtype)
    kctx, vctx = cacheref.contexts(kind)
    scale = 1 / math.sqrt(D)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    pd = None if perm is None else torch.tensor(perm, dtype=torch.int32, device=DEV)
    out, sel = tq.sparse_decode_attention(kctx, vctx, cache.off, q, box, kc, vc, sl, Hkv, max_len, scale, block_table=table,
                                          page_tokens=page, select=select, first=first, last=last, channel_perm=pd)
    assert out.dtype == dtype and sel.shape == (B, Hkv, select)
    assert kctx[0].device_error() == 0
    qn, bn, sel = q.double().cpu().numpy(), box.double().cpu().numpy(), sel.cpu().numpy()
    rep = Hq // Hkv
    ref, tol = np.zeros((B, Hq, D)), np.zeros((B, Hq, D))
    for b in range(B):
        n = -(-lens[b] // page)
        for h in range(Hkv):
            rows = slice(h * rep, (h + 1) * rep)
            want = _pick(qn[b, rows], bn[cache.table[b, :n], h], n, select, first, last)
            assert sel[b, h].tolist() == want.tolist() + [-1] * (select - len(want)), (b, h)
            t = (want[:, None] * page + np.arange(page)).reshape(-1)
            t = t[t < lens[b]]
            if len(t):
                ref[b, rows], tol[b, rows] = cache.attend(b, h, qn[b, rows], t, np.ones((rep, len(t)), bool), scale, perm)
    cacheref.check(out, ref, tol, dtype, "sparse")
    return out


@gpu
@pytest.mark.parametrize("kind", sorted(cacheref.LAYOUTS))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_sparse_matches(kind, dtype):
    _case(1, kind, 3, 8, 2, [700, 0, 129], 64, 4, 1, 1, dtype)


@gpu
@pytest.mark.parametrize("Hq,Hkv,lens,page,select,first,last", [
    (4, 4, [1, 64, 65], 64, 1, 0, 0),             # one head a kv head, one page
    (7, 1, [1000], 128, 3, 2, 2),                 # forced pages outnumber the selection: the lower ones win
    (32, 8, [640, 639], 64, 10, 1, 1),            # every page
    (16, 2, [513], 64, 9, 0, 1),                  # as many as there are, the last one of a single token
    (6, 2, [2000, 1500], 256, 5, 0, 0),
    (5, 1, [64 * 40], 64, 33, 1, 2),
])
def test_sparse_shapes(Hq, Hkv, lens, page, select, first, last):
    _case(2, "4", len(lens), Hq, Hkv, lens, page, select, first, last, torch.bfloat16)


@gpu
def test_sparse_many_pages():
    """More pages than the selection's block has threads, several pages a thread in every pass."""
    _case(3, "2.5", 1, 4, 1, [64 * 700 - 3], 64, 65, 1, 2, torch.bfloat16)


@gpu
@pytest.mark.parametrize("same", [False, True])
def test_sparse_page_counts(same):
    """Page counts around every power of two and every way of selecting, next to one another in one batch."""
    n = [9, 16, 17, 32, 33, 64, 65, 128, 129, 255, 256, 257, 300]
    box = None
    if same:                                      # every score equal: the lower pages
        pool = cacheref.Cache(np.random.default_rng(7), "3", len(n), 1, [64 * x - 5 for x in n], 64 * max(n), 64).pool
        box = torch.ones((pool, 1, 2, D), device=DEV, dtype=torch.bfloat16)
    _case(7, "3", len(n), 2, 1, [64 * x - 5 for x in n], 64, 8, 0 if same else 2, 1, torch.bfloat16, box=box)


@gpu
def test_sparse_ties_infinities_and_nan():
    """Equal scores go to the lower page; infinite bounds win or lose; a NaN score comes last."""
    page, n, Hkv = 64, 12, 1
    rng = np.random.default_rng(4)
    table = rng.permutation(n + 2)[:n].astype(np.int32)     # (as Cache draws it)
    box = np.full((n + 2, 1, 2, D), 0.0)
    box[:, :, 0], box[:, :, 1] = -1.0, 1.0
    box[table[3], 0, 1, 5] = np.inf
    box[table[8], 0, 1, 5], box[table[8], 0, 0, 5] = np.nan, np.nan
    box[table[9], 0, :, 0] = [-1.5, 1.5]
    t = torch.tensor(box, device=DEV).bfloat16()
    _case(4, "4", 1, 4, 1, [n * page], page, 4, 0, 0, torch.bfloat16, box=t)
    _case(4, "4", 1, 4, 1, [n * page], page, 11, 0, 0, torch.bfloat16, box=t)
    same = torch.ones_like(t)
    _case(4, "4", 1, 4, 1, [n * page], page, 5, 0, 1, torch.bfloat16, box=same)


@gpu
def test_sparse_channel_permutation():
    perm = np.stack([np.random.default_rng(h).permutation(D) for h in range(3)]).astype(np.int32)
    _case(5, "2.5", 2, 12, 3, [500, 300], 64, 3, 1, 1, torch.bfloat16, perm=perm)


@gpu
def test_sparse_of_every_page_is_decode_attention():
    rng = np.random.default_rng(6)
    B, Hq, Hkv, page, lens = 2, 8, 2, 64, [300, 77]
    cache = cacheref.Cache(rng, "3.5", B, Hkv, lens, 320, page)
    kc, vc, table = cacheref.upload(cache, DEV)
    kctx, vctx = cacheref.contexts("3.5")
    q = torch.randn(B, Hq, D, device=DEV)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    box = torch.zeros(cache.pool, Hkv, 2, D, device=DEV)
    got, sel = tq.sparse_decode_attention(kctx, vctx, cache.off, q, box, kc, vc, sl, Hkv, 320, 0.1, block_table=table,
                                          page_tokens=page, select=5)
    want = tq.decode_attention(kctx, vctx, cache.off, q, kc, vc, sl, Hkv, 320, 0.1, block_table=table, page_tokens=page)
    assert (got - want).abs().max() <= 1e-5 * want.abs().max()         # the same products, split at other places
    assert sel[0, 0].tolist() == [0, 1, 2, 3, 4] and sel[1, 1].tolist() == [0, 1, -1, -1, -1]


@gpu
def test_sparse_bad_pages_are_reported():
    rng = np.random.default_rng(7)
    cache = cacheref.Cache(rng, "4", 1, 2, [640], 640, 64)
    kc, vc, table = cacheref.upload(cache, DEV)
    kctx, vctx = cacheref.contexts("4")
    q, box = torch.randn(1, 8, D, device=DEV), torch.randn(cache.pool, 2, 2, D, device=DEV).sort(2).values
    sl = torch.tensor([640], dtype=torch.int32, device=DEV)
    table[0, 4], table[0, 9] = 1 << 30, -3
    out, sel = tq.sparse_decode_attention(kctx, vctx, cache.off, q, box, kc, vc, sl, 2, 640, 0.1, block_table=table,
                                          page_tokens=64, select=4, first=0, last=1)
    torch.cuda.synchronize()
    assert kctx[0].device_error() == 901 and sel[0, 0, -1] == 9 and 4 not in sel[0].tolist()[0]


@gpu
def test_sparse_plan_replayed_from_a_graph_and_its_refusals():
    rng = np.random.default_rng(8)
    cache = cacheref.Cache(rng, "4", 2, 2, [640, 200], 640, 64)
    kc, vc, table = cacheref.upload(cache, DEV)
    kctx, vctx = cacheref.contexts("4")
    q, box = torch.randn(2, 8, D, device=DEV).half(), torch.randn(cache.pool, 2, 2, D, device=DEV).half().sort(2).values
    sl = torch.tensor([640, 200], dtype=torch.int32, device=DEV)
    plan = tq.SparsePlan(kctx, vctx, cache.off, kc, vc, 2, 8, 2, D, 640, block_table=table, page_tokens=64, select=3)
    plan(q, box, sl, 0.1)
    out = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan(q, box, sl, 0.1, out=out)
    q.copy_(torch.randn_like(q))
    sl.copy_(torch.tensor([130, 600], dtype=torch.int32))
    graph.replay()
    got, sel = out.clone(), plan.selected.clone()
    want, wsel = plan(q, box, sl, 0.1)
    assert torch.equal(got, want) and torch.equal(sel, wsel)
    for bad in (lambda: plan(q[:1], box, sl, 0.1), lambda: plan(q, box[:, :1], sl, 0.1), lambda: plan(q, box, sl.long(), 0.1),
                lambda: plan(q, box.cpu(), sl, 0.1), lambda: plan(q, box, sl, 0.1, out=out.float()),
                lambda: tq.SparsePlan(kctx, vctx, cache.off, kc, vc, 2, 8, 2, D, 640, block_table=table[:1], page_tokens=64, select=3)):
        with pytest.raises(ValueError):
            bad()
    plan.workspace = plan.workspace[:16]
    with pytest.raises(tq.TQError) as e:
        plan(q, box, sl, 0.1)
    assert e.value.status == 5

"""tq_tree_attention: drafted tokens over the packed cache, against the definition in 64 bits."""
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


# ------------------------------------------------------------------ host
def test_tree_mask_is_the_ancestors():
    rng = np.random.default_rng(0)
    for T in (1, 5, 64, 65, 200):
        p = np.array([[rng.integers(-1, j) for j in range(T)] for _ in range(3)], dtype=np.int32)
        m = tq.tree_mask(p)
        assert m.shape == (3, T, -(-T // 64)) and m.dtype == np.int64
        for b in range(3):
            for j in range(T):
                up, anc = j, set()
                while up >= 0:
                    anc.add(up)
                    up = p[b, up]
                bits = {64 * w + i for w in range(m.shape[2]) for i in range(64) if int(m[b, j, w]) >> i & 1}
                assert bits == anc
    assert tq.tree_mask([-1, 0, 0]).tolist() == [[[1], [3], [5]]]


@pytest.mark.parametrize("p", [[0], [-1, 1], [-2], [-1, 0, 5]])
def test_tree_mask_refuses(p):
    with pytest.raises(tq.TQError) as e:
        tq.tree_mask(p)
    assert e.value.status == 1


def test_tree_refusals_without_gpu():
    L = tq.lib()
    assert tq.tree_workspace_size(1, 0, 8, 2, D, 1, 100) == 0 and tq.tree_workspace_size(1, 257, 8, 2, D, 1, 100) == 0
    assert tq.tree_workspace_size(1, 4, 8, 3, D, 1, 100) == 0 and tq.tree_workspace_size(1, 4, 8, 2, 64, 1, 100) == 0
    assert tq.tree_workspace_size(1, 4, 8, 2, D, 1, 100) > 0
    o = tq._DecodeOpts(0, 4096, 96)
    args = [None, None, None, 1, None, 1, None, None, None, None, None, 1, 4, 8, 2, D, 192, 1.0, None]
    assert L.tq_tree_attention(*args, None, None, 0, None) == 1
    args[12] = 257
    assert L.tq_tree_attention(*args, None, None, 0, None) == 2
    args[12] = 4
    assert L.tq_tree_attention(*args, ctypes.byref(o), None, 0, None) == 1       # a page of 96 tokens


# ------------------------------------------------------------------ GPU
def _random_tree(rng, B, T):
    return np.array([[rng.integers(-1, j) if j else -1 for j in range(T)] for _ in range(B)], dtype=np.int32)


def _keep(mask, b, j, n, words):
    return np.array([(int(mask[b, j, i // 64]) >> (i % 64)) & 1 for i in range(n)], bool)


def _reference(cache, q, lens, drafts, mask, scale, perm=None):
    B, T, Hq, _ = q.shape
    Hkv = cache.Hkv
    rep = Hq // Hkv
    ref, tol = np.zeros(q.shape), np.zeros(q.shape)
    for b in range(B):
        L = min(max(lens[b], 0), cache.max_len)
        n = min(T, L) if drafts is None else max(0, min(drafts[b], T, L))
        if not n:
            continue
        keep = np.ones((n, L), bool)
        for j in range(n):
            keep[j, L - n:] = _keep(mask, b, j, n, 0) if mask is not None else np.arange(n) <= j
        for h in range(Hkv):
            rows = q[b, :n, h * rep:(h + 1) * rep].reshape(n * rep, D)
            o, t = cache.attend(b, h, rows, np.arange(L), np.repeat(keep, rep, 0), scale, perm)
            ref[b, :n, h * rep:(h + 1) * rep] = o.reshape(n, rep, D)
            tol[b, :n, h * rep:(h + 1) * rep] = t.reshape(n, rep, D)
    return ref, tol


def _case(seed, kind, Hq, Hkv, T, lens, drafts, dtype=torch.bfloat16, page=0, max_len=None, mask="tree", perm=None,
          scale=1 / math.sqrt(D), spread=0.5, qscale=1.0, edit=None):
    rng = np.random.default_rng(seed)
    B = len(lens)
    most = max(max(lens), 1)
    max_len = max_len or (-(-most // page) * page if page else most)
    cache = cacheref.Cache(rng, kind, B, Hkv, [min(max(n, 0), max_len) for n in lens], max_len, page, spread=spread)
    if edit:
        edit(cache)
    kc, vc, table = cacheref.upload(cache, DEV)
    q = torch.tensor(qscale * rng.standard_normal((B, T, Hq, D)), device=DEV).to(dtype)
    m = tq.tree_mask(_random_tree(rng, B, T)) if isinstance(mask, str) else mask
    i32 = lambda v: None if v is None else torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    kctx, vctx = cacheref.contexts(kind)
    out = tq.tree_attention(kctx, vctx, cache.off, q, kc, vc, i32(lens), Hkv, max_len, scale, i32(drafts),
                            None if m is None else torch.tensor(m, device=DEV), channel_perm=i32(perm), block_table=table,
                            page_tokens=page)
    torch.cuda.synchronize()
    assert kctx[0].device_error() == 0 and out.dtype == dtype
    ref, tol = _reference(cache, q.double().cpu().numpy(), lens, drafts, m, scale, perm)
    cacheref.check(out, ref, tol, dtype, "tree")
    return out, ref


@gpu
@pytest.mark.parametrize("kind", sorted(cacheref.LAYOUTS))
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_tree_matches(kind, dtype):
    _case(1, kind, 8, 2, 6, [200, 65, 131], [6, 3, 5], dtype, page=64)


@gpu
@pytest.mark.parametrize("Hq,Hkv,T,lens,drafts,page", [
    (4, 4, 1, [1, 64, 65], [1, 1, 1], 0),                # single drafted tokens, one query head a kv head
    (8, 1, 3, [3, 2, 1, 0], [3, 2, 1, 0], 0),            # nothing but drafts; an empty sequence
    (7, 1, 23, [300], [23], 128),                        # 161 rows a kv head: two row blocks, an odd last row
    (32, 8, 16, [190, 77], [16, 9], 64),                 # 64 rows
    (5, 1, 64, [257], [64], 0),                          # 320 rows; drafts across a tile border
    (2, 2, 200, [333, 201], [200, 130], 64),             # masks of four words
    (16, 1, 9, [1000, 3], [9, 3], 256),                  # 144 rows, splits
    (6, 2, 40, [40, 41, 100], None, 0),                  # every sequence drafts T
    (1, 1, 256, [256, 300], [256, 255], 0),              # the most drafts
])
def test_tree_shapes(Hq, Hkv, T, lens, drafts, page):
    _case(2, "4", Hq, Hkv, T, lens, drafts, page=page)


@gpu
def test_tree_long_context_in_many_splits():
    _case(3, "2.5", 4, 1, 12, [9000], [12], page=64)
    _case(3, "3.5", 4, 1, 12, [8191, 30], [12, 12], max_len=8192)


@gpu
@pytest.mark.parametrize("T", [2, 5, 9, 17])
@pytest.mark.parametrize("kind", ["4", "2.5"])
def test_tree_many_tiles_a_block(T, kind):
    """So many kv heads that a block runs through 1 to 11 tiles: every phase of its pipeline, in each fold of the rows."""
    lens = [64 * i + (i % 3) for i in range(1, 12)]
    _case(16, kind, 4 * 16, 16, T, lens, [T] * 11, page=64)


@gpu
def test_tree_odd_cache_lengths():
    """Sequences start at odd slots, so records and norms sit at odd offsets."""
    _case(4, "3.5", 12, 3, 5, [257, 130], [5, 5], max_len=257)
    _case(4, "3", 12, 3, 5, [255, 1], [5, 1], max_len=255)


@gpu
def test_tree_chain_and_lengths_that_are_clamped():
    _case(5, "4", 8, 2, 7, [100, 5, 400], [7, 9, -3], mask=None, max_len=300)
    out, _ = _case(5, "4", 8, 2, 7, [100, -5], [0, 7], mask=None)
    assert (out == 0).all()


@gpu
def test_tree_rows_that_attend_nothing():
    """Without a context, a row whose mask is empty gives zeros; other rows of its block are not touched by it."""
    T = 6
    m = np.zeros((2, T, 1), dtype=np.int64)
    m[0, 1], m[0, 3], m[1, :, 0] = 2, 0b111111, -1
    out, _ = _case(6, "4", 8, 2, T, [6, 70], [6, 6], mask=m)
    assert (out[0, [0, 2, 4, 5]] == 0).all() and (out[0, 1] != 0).any()


@gpu
def test_tree_mask_bits_past_the_drafts_are_ignored():
    m = np.full((1, 5, 1), -1, dtype=np.int64)
    _case(7, "4", 8, 2, 5, [80], [3], mask=m)


@gpu
def test_tree_channel_permutation():
    perm = np.stack([np.random.default_rng(h).permutation(D) for h in range(3)]).astype(np.int32)
    _case(8, "2.5", 12, 3, 5, [150, 90], [5, 4], perm=perm, page=64)


@gpu
@pytest.mark.parametrize("qscale,spread", [(20.0, 0.5), (1e-3, 2.0), (1.0, 0.0)])
def test_tree_peaked_and_flat_weights(qscale, spread):
    """Logits of hundreds (the running maximum moves on), and of nearly nothing under very unequal values."""
    _case(9, "3.5", 8, 2, 8, [700], [8], torch.float32, qscale=qscale, spread=spread)


@gpu
def test_tree_growing_maxima():
    """Keys that grow along the context: every tile raises the maximum."""
    def grow(cache):
        for t in range(cache.lens[0]):
            cache.set_norms(0, t, key=np.float16(0.5 + 0.2 * t))
    _case(10, "4", 4, 1, 4, [400], [4], torch.float32, edit=grow)
    def fall(cache):
        for t in range(cache.lens[0]):
            cache.set_norms(0, t, key=np.float16(0.5 + 0.2 * (400 - t)))
    _case(10, "4", 4, 1, 4, [400], [4], torch.float32, edit=fall)


@gpu
def test_tree_large_and_zero_norms():
    def edit(cache):
        cache.set_norms(0, 3, key=np.float16(0.0), value=np.float16(0.0))
        cache.set_norms(0, 17, value=np.float16(60000.0))
        cache.set_norms(0, 20, value=np.float16(3e-5))
    _case(11, "4", 8, 2, 4, [90], [4], torch.float32, edit=edit)


@gpu
@pytest.mark.parametrize("kind", ["4", "2.5"])
@pytest.mark.parametrize("which", ["key", "value"])
def test_tree_norms_that_are_not_finite_stay_with_the_rows_that_attend_them(kind, which):
    """Drafted tokens 2 (infinite) and 4 (NaN): only rows that attend one of them are NaN."""
    T, lens = 6, [150]
    m = tq.tree_mask([[-1, 0, 0, 1, 2, 3]])                        # rows 2 and 4 attend token 2, row 4 token 4 too
    bad = [2, 4]

    def edit(cache, values):
        for t, v in zip(bad, values):
            cache.set_norms(0, 144 + t, **{which: np.float16(v)})

    out, _ = _case(17, kind, 8, 2, T, lens, [T], mask=m, edit=lambda c: edit(c, (1.0, 1.0)))
    rng = np.random.default_rng(17)
    cache = cacheref.Cache(rng, kind, 1, 2, lens, 150)
    edit(cache, (np.inf, np.nan))
    kc, vc, _ = cacheref.upload(cache, DEV)
    q = torch.tensor(rng.standard_normal((1, T, 8, D)), device=DEV).bfloat16()
    kctx, vctx = cacheref.contexts(kind)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    got = tq.tree_attention(kctx, vctx, cache.off, q, kc, vc, i32(150), 2, 150, 1 / math.sqrt(D), i32(T), torch.tensor(m, device=DEV))
    fine = [0, 1, 3, 5]
    assert torch.equal(got[0, fine], out[0, fine])
    if which == "value":
        assert got[0, bad].isnan().all()
    else:
        assert not got[0, bad].isfinite().all()


@gpu
def test_tree_waits_that_run_out_are_reported():
    """The products wait for a barrier that nothing arrives on: after a millisecond the kernel gives up, says so and
    winds down, and the next call is right again."""
    rng = np.random.default_rng(18)
    cache = cacheref.Cache(rng, "4", 2, 2, [500, 300], 512, 64)
    kc, vc, table = cacheref.upload(cache, DEV)
    kctx, vctx = cacheref.contexts("4")
    q = torch.randn(2, 4, 8, D, device=DEV).bfloat16()
    sl = torch.tensor([500, 300], dtype=torch.int32, device=DEV)
    plan = tq.TreePlan(kctx, vctx, cache.off, kc, vc, 2, 4, 8, 2, D, 512, block_table=table, page_tokens=64)
    want = plan(q, sl, None, None, 0.1)
    torch.cuda.synchronize()
    assert kctx[0].device_error() == 0
    try:
        tq.lib().tq_debug_set_wait_limit(1000000)
        tq.lib().tq_debug_inject_stall(1)
        plan(q, sl, None, None, 0.1)
        torch.cuda.synchronize()
    finally:
        tq.lib().tq_debug_inject_stall(0)
        tq.lib().tq_debug_set_wait_limit(2000000000)
    assert 601 <= kctx[0].device_error() <= 615
    assert torch.equal(plan(q, sl, None, None, 0.1), want) and kctx[0].device_error() == 0


@gpu
def test_tree_of_one_token_is_decode_attention():
    rng = np.random.default_rng(12)
    lens = [300, 77, 1]
    cache = cacheref.Cache(rng, "3.5", 3, 2, lens, 320, 64)
    kc, vc, table = cacheref.upload(cache, DEV)
    kctx, vctx = cacheref.contexts("3.5")
    q = torch.randn(3, 8, D, device=DEV)
    sl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    kw = dict(block_table=table, page_tokens=64)
    got = tq.tree_attention(kctx, vctx, cache.off, q[:, None], kc, vc, sl, 2, 320, 0.1, **kw)[:, 0]
    want = tq.decode_attention(kctx, vctx, cache.off, q, kc, vc, sl, 2, 320, 0.1, **kw)
    ref, tol = _reference(cache, q[:, None].double().cpu().numpy(), lens, None, None, 0.1)
    cacheref.check(got, ref[:, 0], tol[:, 0], torch.float32)
    cacheref.check(want, ref[:, 0], tol[:, 0], torch.float32)


@gpu
def test_tree_bad_page_is_reported():
    rng = np.random.default_rng(13)
    cache = cacheref.Cache(rng, "4", 1, 2, [300], 320, 64)
    kc, vc, table = cacheref.upload(cache, DEV)
    kctx, vctx = cacheref.contexts("4")
    table[0, 2] = 1 << 28
    q = torch.randn(1, 3, 8, D, device=DEV)
    tq.tree_attention(kctx, vctx, cache.off, q, kc, vc, torch.tensor([300], dtype=torch.int32, device=DEV), 2, 320, 0.1,
                      block_table=table, page_tokens=64)
    torch.cuda.synchronize()
    assert kctx[0].device_error() == 901


@gpu
def test_calls_on_another_stream_own_what_they_allocate():
    """Queries that are not contiguous, outputs and workspaces of calls on a side stream, with the current stream
    busy reusing memory at the same time; tables on the host are refused before anything runs."""
    rng = np.random.default_rng(24)
    cache = cacheref.Cache(rng, "4", 2, 2, [200, 90], 256, 64)
    kc, vc, table = cacheref.upload(cache, DEV)
    kctx, vctx = cacheref.contexts("4")
    wide = torch.randn(2, 5, 8, 2 * D, device=DEV).bfloat16()
    q, q1 = wide[..., :D], wide[:, 0, :, D:]
    box = torch.randn(cache.pool, 2, 2, D, device=DEV).bfloat16().sort(2).values
    sl = torch.tensor([200, 90], dtype=torch.int32, device=DEV)
    args = (kctx, vctx, cache.off)
    tree = lambda **kw: tq.tree_attention(*args, q, kc, vc, sl, 2, 256, 0.1, block_table=table, page_tokens=64, **kw)  # noqa: E731
    sparse = lambda **kw: tq.sparse_decode_attention(*args, q1, box, kc, vc, sl, 2, 256, 0.1, block_table=table,  # noqa: E731
                                                     page_tokens=64, select=2, **kw)
    pos, f = torch.arange(10, device=DEV), torch.ones(64, dtype=torch.float64, device=DEV)
    rows = wide.reshape(10, 8, 2 * D)[..., :D]
    want_t, (want_s, want_p), (want_r, _) = tree(), sparse(), tq.rope(rows, None, pos, f)
    side = torch.cuda.Stream()
    for _ in range(20):
        side.wait_stream(torch.cuda.current_stream())
        t, (s, p), (r, _) = tree(stream=side), sparse(stream=side), tq.rope(rows, None, pos, f, stream=side)
        for _ in range(4):
            torch.full((1 << 16,), float("nan"), device=DEV)
            torch.full((2, 5, 8, D), float("nan"), device=DEV, dtype=torch.bfloat16)
        side.synchronize()
        assert torch.equal(t, want_t) and torch.equal(s, want_s) and torch.equal(p, want_p) and torch.equal(r, want_r)
    with pytest.raises(ValueError):
        tq.tree_attention(*args, q, kc, vc, sl, 2, 256, 0.1, block_table=table.cpu(), page_tokens=64)
    with pytest.raises(ValueError):
        tq.sparse_decode_attention(*args, q1, box, kc, vc, sl, 2, 256, 0.1, block_table=table.cpu(), page_tokens=64, select=2)
    with pytest.raises(ValueError):
        tree(channel_perm=torch.arange(D, dtype=torch.int32).repeat(2, 1))
    with pytest.raises(ValueError):
        tq.rope(rows, None, pos, f, q_out=torch.empty(10, 1, D, device=DEV, dtype=torch.bfloat16).expand(10, 8, D))


@gpu
def test_tree_plan_streams_graphs_and_refusals():
    rng = np.random.default_rng(14)
    cache = cacheref.Cache(rng, "4", 2, 2, [200, 90], 256, 64)
    kc, vc, table = cacheref.upload(cache, DEV)
    kctx, vctx = cacheref.contexts("4")
    T = 5
    q = torch.randn(2, T, 8, D, device=DEV).bfloat16()
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    sl, dl = i32(200, 90), i32(5, 3)
    mask = torch.tensor(tq.tree_mask(_random_tree(rng, 2, T)), device=DEV)
    plan = tq.TreePlan(kctx, vctx, cache.off, kc, vc, 2, T, 8, 2, D, 256, block_table=table, page_tokens=64)
    want = plan(q, sl, dl, mask, 0.1)
    out = torch.full_like(q, float("nan"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    plan(q, sl, dl, mask, 0.1, out=out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    assert torch.equal(plan(q, sl, dl, mask, 0.1), want)                 # the same bits every time
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan(q, sl, dl, mask, 0.1, out=out)
    q.copy_(torch.randn_like(q))
    sl.copy_(i32(64, 200))
    dl.copy_(i32(1, 5))
    graph.replay()
    got = out.clone()                                       # (sequence 1 now reads unused slots: NaN on both sides)
    assert torch.allclose(got, plan(q, sl, dl, mask, 0.1), rtol=0, atol=0, equal_nan=True) and not got[0].isnan().any()
    sl.copy_(i32(130, 88))
    graph.replay()
    got = out.clone()
    assert torch.equal(got, plan(q, sl, dl, mask, 0.1)) and not got.isnan().any()
    for bad in (lambda: plan(q[:, :4], sl, dl, mask, 0.1), lambda: plan(q, sl.long(), dl, mask, 0.1),
                lambda: plan(q, sl, dl[:1], mask, 0.1), lambda: plan(q, sl, dl, mask.int(), 0.1),
                lambda: plan(q, sl, dl, mask[:, :, 0], 0.1), lambda: plan(q, sl, dl, mask, 0.1, out=out.float()),
                lambda: plan(q, sl.cpu(), dl, mask, 0.1)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        plan(q.double(), sl, dl, mask, 0.1)
    plan.workspace = plan.workspace[:16]
    with pytest.raises(tq.TQError) as e:
        plan(q, sl, dl, mask, 0.1)
    assert e.value.status == 5
    for T in (0, 257):
        big = torch.zeros(2, T, 8, D, device=DEV)
        with pytest.raises(tq.TQError) as e:
            tq.tree_attention(kctx, vctx, cache.off, big, kc, vc, sl, 2, 256, 0.1, block_table=table, page_tokens=64)
        assert e.value.status == 2
    other, _ = tq.Context(128, 5, 1, tq.MODE_PROD), None
    with pytest.raises(tq.TQError) as e:                                  # 5-bit keys: no decode kernel reads them
        tq.tree_attention([other], vctx, cache.off, q, [tq.alloc_packed(other, kc[0].cap)], vc, sl, 2, 256, 0.1,
                          block_table=table, page_tokens=64)
    assert e.value.status == 2


@gpu
@pytest.mark.parametrize("perm", [False, True])
def test_a_serving_step_end_to_end(perm):
    """Prompt, then drafted tokens: rotate, quantize into the paged cache, keep the page bounds, verify the drafts, and
    attend over selected pages; every stage against 64 bits on what the stage before it stored."""
    kind, B, Hq, Hkv, page, T = "3.5", 2, 8, 2, 64, 4
    rng = np.random.default_rng(15)
    lens, max_len = [200, 130], 256
    cache = cacheref.Cache(rng, kind, B, Hkv, lens, max_len, page, poison=False)
    kc, vc, table = cacheref.upload(cache, DEV)
    kctx, vctx = cacheref.contexts(kind)
    gen = torch.Generator(device=DEV).manual_seed(1)
    n = B * T
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
    freq, factor = tq.rope_frequencies(D, 500000.0, "bands", factor=8.0, original_len=8192, low=1.0, high=4.0)
    q = torch.randn(n, Hq, D, generator=gen, device=DEV).bfloat16()
    k = torch.randn(n, Hkv, D, generator=gen, device=DEV).bfloat16()
    v = torch.randn(n, Hkv, D, generator=gen, device=DEV).bfloat16()
    parents = _random_tree(rng, B, T)
    depth = np.zeros((B, T), int)
    for b in range(B):
        for j in range(T):
            depth[b, j] = 0 if parents[b, j] < 0 else depth[b, parents[b, j]] + 1
    start = [x - T for x in lens]
    pos = i32([[s + int(d) for d in row] for s, row in zip(start, depth)]).reshape(-1)
    q, k = tq.rope(q, k, pos, torch.tensor(freq, device=DEV), factor=factor)
    slots = torch.tensor(np.stack([[cache.slots(b, h, np.array([start[b] + j]))[0] for h in range(Hkv)]
                                   for b in range(B) for j in range(T)]), device=DEV).reshape(-1)
    cp = None
    if perm:
        cp = np.stack([np.random.default_rng(h).permutation(D) for h in range(Hkv)]).astype(np.int32)
    for g, (w, kb, vb) in enumerate(cache.groups):
        for x, ctx, store, pk in ((k, kctx[g], cache.k[g], kc[g]), (v, vctx[g], cache.v[g], vc[g])):
            if perm:
                for h in range(Hkv):
                    tq.quantize_kv(ctx, x[:, h].contiguous(), pk, slots=slots.reshape(n, Hkv)[:, h].contiguous(),
                                   cols=i32(cp[h, cache.off[g]:cache.off[g + 1]]))
            else:
                tq.quantize_kv(ctx, x.reshape(n * Hkv, D)[:, cache.off[g]:cache.off[g + 1]], pk, slots=slots)
            import layout
            store["codes"] = pk.codes.cpu().numpy()
            store["idx"], store["signs"], _ = layout.unpack(store["codes"], w, ctx.k, ctx.mode == 0)
            store["norm"] = pk.norm.cpu().numpy()
            store["rnorm"] = None if pk.rnorm is None else pk.rnorm.cpu().numpy()
    bounds = torch.randn(cache.pool, Hkv, 2, D, generator=gen, device=DEV).sort(2).values.bfloat16()
    tq.page_bounds(k, i32([0, T, 2 * T]), i32(start), table, page, bounds, T)
    mask = tq.tree_mask(parents)
    scale = 1 / math.sqrt(D)
    out = tq.tree_attention(kctx, vctx, cache.off, q.reshape(B, T, Hq, D), kc, vc, i32(lens), Hkv, max_len, scale,
                            mask=torch.tensor(mask, device=DEV), block_table=table, page_tokens=page,
                            channel_perm=None if cp is None else i32(cp))
    ref, tol = _reference(cache, q.reshape(B, T, Hq, D).double().cpu().numpy(), lens, None, mask, scale, cp)
    cacheref.check(out, ref, tol, torch.bfloat16, "tree")
    last = q.reshape(B, T, Hq, D)[:, -1]
    got, sel = tq.sparse_decode_attention(kctx, vctx, cache.off, last.contiguous(), bounds, kc, vc, i32(lens), Hkv, max_len,
                                          scale, block_table=table, page_tokens=page, select=2,
                                          channel_perm=None if cp is None else i32(cp))
    ln, sel, rep = last.double().cpu().numpy(), sel.cpu().numpy(), Hq // Hkv
    for b in range(B):
        for h in range(Hkv):
            assert sel[b, h].tolist()[0] == 0 and sel[b, h].tolist()[1] == -(-lens[b] // page) - 1
            t = (sel[b, h][:, None] * page + np.arange(page)).reshape(-1)
            t = t[t < lens[b]]
            o, tl = cache.attend(b, h, ln[b, h * rep:(h + 1) * rep], t, np.ones((rep, len(t)), bool), scale, cp)
            cacheref.check(got[b, h * rep:(h + 1) * rep], o, tl, torch.bfloat16, "sparse")

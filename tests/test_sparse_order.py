"""tq_sparse_decode_attention: steps behind one another read the lengths and pages of their own selection."""
import numpy as np
import pytest

import cacheref
import kv_cache_vector_08_b200 as tq

torch = pytest.importorskip("torch")
gpu = pytest.mark.gpu
DEV = torch.device("cuda", 0)
D = 128


@gpu
@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("kind,pages,select", [("3.5", 12, 5), ("4", 200, 7), ("2.5", 6, 6)])
def test_steps_in_a_row_attend_their_own_selection(kind, pages, select, captured):
    """The decode kernel of a step starts before the memory of the selection in front is visible to it.  Twenty steps
    of other queries and lengths run without a wait in between, the workspace filled with values that no selection
    writes: a length or page of an earlier step, or of the filling, gives other outputs or a bad page.  Each step is
    then attended again by tq_decode_attention, which does not start so, over the pages that the step says it took:
    the same kernel on the same split of the same tokens, so bit by bit."""
    rng = np.random.default_rng(pages)
    B, Hq, Hkv, page, steps = 3, 8, 2, 64, 20
    max_len, rep = pages * page, Hq // Hkv
    cache = cacheref.Cache(rng, kind, B, Hkv, [max_len] * B, max_len, page)
    kc, vc, table = cacheref.upload(cache, DEV)
    kctx, vctx = cacheref.contexts(kind)
    gen = torch.Generator(device=DEV).manual_seed(pages)
    q = torch.randn(steps, B, Hq, D, generator=gen, device=DEV)
    box = torch.randn(cache.pool, Hkv, 2, D, generator=gen, device=DEV).sort(2).values
    lens = torch.tensor(rng.integers(1, max_len + 1, (steps, B)), dtype=torch.int32, device=DEV)
    plan = tq.SparsePlan(kctx, vctx, cache.off, kc, vc, B, Hq, Hkv, D, max_len, block_table=table, page_tokens=page, select=select)
    outs, sels = torch.empty(steps, B, Hq, D, device=DEV), torch.empty(steps, B, Hkv, select, dtype=torch.int32, device=DEV)

    def run():
        for i in range(steps):
            plan.workspace.fill_(0x7F)
            plan(q[i], box, lens[i], 0.1, out=outs[i])
            sels[i] = plan.selected

    run()
    if captured:
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            run()
        outs.zero_()
        for _ in range(3):
            graph.replay()
    torch.cuda.synchronize()
    assert kctx[0].device_error() == 0
    heads = torch.arange(Hkv, device=DEV, dtype=torch.int32)[None, :, None]
    for i in range(steps):
        sel, n = sels[i], lens[i][:, None, None]
        phys = torch.gather(table[:, None].expand(B, Hkv, pages), 2, sel.clamp(min=0).long()) * Hkv + heads
        tokens = ((n - sel * page).clamp(max=page) * (sel >= 0)).sum(2).to(torch.int32)
        assert (sel[:, :, 0] >= 0).all()
        want = tq.decode_attention(kctx, vctx, cache.off, q[i].reshape(B * Hkv, rep, D), kc, vc, tokens.reshape(-1), 1,
                                   select * page, 0.1, block_table=phys.to(torch.int32).reshape(B * Hkv, select).contiguous(),
                                   page_tokens=page)
        assert torch.equal(outs[i], want.reshape(B, Hq, D)), i
    assert kctx[0].device_error() == 0

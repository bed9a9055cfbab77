"""Plans of the calls around the cache: their own memory on the streams that use it."""
import contextlib
import types

import pytest

import cacheref
import kv_cache_vector_08_b200 as tq

torch = pytest.importorskip("torch")
gpu = pytest.mark.gpu
DEV = torch.device("cuda", 0)
D = 128


class _Stream:
    def __init__(self, raw):
        self.cuda_stream = raw


@pytest.fixture
def host(monkeypatch):
    """The binding with a library that takes every call, streams by number and a log of record_stream."""
    fake = types.SimpleNamespace(tq_sparse_workspace_size=lambda *a: 256, tq_tree_workspace_size=lambda *a: 512,
                                 tq_sparse_decode_attention=lambda *a: 0, tq_tree_attention=lambda *a: 0)
    state = types.SimpleNamespace(current=_Stream(11), log=[])
    monkeypatch.setattr(tq, "lib", lambda: fake)
    monkeypatch.setattr(tq, "_raw_stream", lambda stream: (state.current if stream is None else stream).cuda_stream)
    monkeypatch.setattr(tq, "_on_current_device", lambda *t: None)
    monkeypatch.setattr(tq, "_on", lambda stream: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: state.current)
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: state.log.append((t.data_ptr(), s.cuda_stream)))
    return state


def _caches():
    ctx = types.SimpleNamespace(handle=types.SimpleNamespace(value=1))
    pk = tq.Packed(torch.zeros(4, 8, dtype=torch.uint8), torch.zeros(4).half(), torch.zeros(4).half())
    return [ctx], [ctx], [0, D], [pk], [pk]


@pytest.mark.parametrize("which", ["sparse", "tree"])
def test_own_memory_is_recorded_on_every_other_stream(host, which):
    i32 = torch.zeros(1, dtype=torch.int32)
    if which == "sparse":
        plan = tq.SparsePlan(*_caches(), 1, 2, 1, D, 64, block_table=i32[None], page_tokens=64, select=1)
        q, bounds = torch.zeros(1, 2, D), torch.zeros(1, 1, 2, D)
        call, own = lambda **kw: plan(q, bounds, i32, 0.1, **kw), [plan.workspace, plan.selected]  # noqa: E731
    else:
        plan = tq.TreePlan(*_caches(), 1, 3, 2, 1, D, 64)
        q = torch.zeros(1, 3, 2, D)
        call, own = lambda **kw: plan(q, i32, None, None, 0.1, **kw), [plan.workspace]  # noqa: E731
    call()
    assert host.log == []                                    # the stream that it was made on
    host.current = _Stream(22)
    call()
    assert host.log == [(t.data_ptr(), 22) for t in own]     # another current stream
    call()
    call(stream=_Stream(11))
    assert len(host.log) == len(own)                         # known already
    call(stream=_Stream(33))
    assert host.log[len(own):] == [(t.data_ptr(), 33) for t in own]


@gpu
def test_a_plan_dropped_while_its_call_runs_on_another_current_stream():
    """The call waits behind other work of the side stream; meanwhile the plan is gone and the stream that it was made
    on fills what memory it gets."""
    import numpy as np
    cache = cacheref.Cache(np.random.default_rng(5), "4", 2, 2, [500, 300], 512, 64)
    kc, vc, table = cacheref.upload(cache, DEV)
    kctx, vctx = cacheref.contexts("4")
    args = (kctx, vctx, cache.off, kc, vc, 2)
    sl = torch.tensor([500, 300], dtype=torch.int32, device=DEV)
    q, qt = torch.randn(2, 8, D, device=DEV), torch.randn(2, 3, 8, D, device=DEV)
    box = torch.randn(cache.pool, 2, 2, D, device=DEV).sort(2).values
    sparse = lambda: tq.SparsePlan(*args, 8, 2, D, 512, block_table=table, page_tokens=64, select=3)  # noqa: E731
    tree = lambda: tq.TreePlan(*args, 3, 8, 2, D, 512, block_table=table, page_tokens=64)  # noqa: E731
    want_s, want_t = sparse()(q, box, sl, 0.1)[0], tree()(qt, sl, None, None, 0.1)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    for _ in range(5):
        a, b = sparse(), tree()
        sizes = [a.workspace.numel(), a.selected.numel() * 4, b.workspace.numel()]
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(4000000)                       # about two milliseconds
            s, t = a(q, box, sl, 0.1)[0], b(qt, sl, None, None, 0.1)
        del a, b
        junk = [torch.full((n,), 0x7F, dtype=torch.uint8, device=DEV) for n in sizes for _ in range(3)]
        torch.cuda.synchronize()
        assert torch.equal(s, want_s) and torch.equal(t, want_t) and kctx[0].device_error() == 0
        del junk


class _On:
    """A tensor that says it is on another GPU."""

    def __init__(self, t, index):
        self.t, self.device = t, torch.device("cuda", index)

    def __getattr__(self, name):
        return getattr(self.t, name)

    def get_device(self):
        return self.device.index


@pytest.mark.parametrize("which", ["sparse", "tree"])
def test_caches_of_another_device_are_refused(monkeypatch, which):
    """Caches of which one lies elsewhere, and a call with another device current than the caches': before anything
    runs."""
    monkeypatch.setattr(tq, "lib", lambda: types.SimpleNamespace(tq_sparse_workspace_size=lambda *a: 256,
                                                                 tq_tree_workspace_size=lambda *a: 256))
    monkeypatch.setattr(tq, "_raw_stream", lambda stream: 0)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    i32 = _On(torch.zeros(1, dtype=torch.int32), 0)
    table = torch.zeros(1, 1, dtype=torch.int32)
    q, bounds = _On(torch.zeros(1, 2, D), 0), _On(torch.zeros(1, 1, 2, D), 0)
    qt = _On(torch.zeros(1, 3, 2, D), 0)

    def plan(*args):
        if which == "sparse":
            return tq.SparsePlan(*args, 1, 2, 1, D, 64, block_table=table, page_tokens=64, select=1)
        return tq.TreePlan(*args, 1, 3, 2, 1, D, 64)

    for i in (3, 4):
        for part in ("codes", "norm", "rnorm"):
            args = _caches()
            setattr(args[i][0], part, _On(getattr(args[i][0], part), 1))
            with pytest.raises(ValueError):
                plan(*args)
    p = plan(*_caches())                                        # (on the host: not on the current device)
    with pytest.raises(ValueError, match="cpu"):
        if which == "sparse":
            p(q, bounds, i32, 0.1, out=_On(torch.zeros(1, 2, D), 0))
        else:
            p(qt, i32, None, None, 0.1, out=_On(torch.zeros(1, 3, 2, D), 0))

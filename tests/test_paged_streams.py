"""Paged-cache calls on other streams than the one a plan was uploaded on."""
import numpy as np
import pytest
import torch

bd = pytest.importorskip("block_causal_varlen_gb300")
pu = pytest.importorskip("paged_util")
paged = bd.paged


class Stream:
    def __init__(self, raw):
        self.cuda_stream = raw


class Memory:
    """Stands in for a plan's device copy: remembers which streams the allocator is told of."""

    def __init__(self):
        self.seen = []

    def record_stream(self, s):
        self.seen.append(s.cuda_stream)


def _uploaded(monkeypatch):
    """A plan as if uploaded on raw stream 0 of device 0, and calls that launch nothing."""
    plan = bd.PagedPlan([1], [20], [[0, 1]], 4, 2, 64, page_size=16, num_pages=3)
    plan.dev, plan._dev_ptr, plan._index, plan._own, plan._streams = Memory(), 64, 0, True, {0}
    now = Stream(0)
    monkeypatch.setattr(paged, "_raw_stream", lambda i: now.cuda_stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: now)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(paged, "_device", lambda *a: 0)
    monkeypatch.setattr(paged, "_rows3", lambda *a: b"")
    monkeypatch.setattr(paged, "_entry", lambda n: lambda *a: 0)
    cache = bd.PagedCache(*(torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16) for _ in range(2)))
    ws = type("Workspace", (), dict(get_device=lambda s: 0, is_contiguous=lambda s: True, data_ptr=lambda s: 256,
                                    numel=lambda s: 1, element_size=lambda s: 1))()
    return plan, now, [lambda **k: bd.bd_cache_write(plan, None, None, cache, **k),
                       lambda **k: bd.bd_cache_read(plan, cache, None, None, **k),
                       lambda **k: bd.bd_paged_attn(plan, None, cache, None, workspace=ws, **k)]


@pytest.mark.parametrize("which", range(3))
def test_a_plans_memory_is_known_to_be_used_on_other_streams(which, monkeypatch):
    plan, now, calls = _uploaded(monkeypatch)
    calls[which]()
    assert plan.dev.seen == []                      # the stream of its upload
    calls[which](stream=Stream(5))
    calls[which](stream=Stream(5))
    assert plan.dev.seen == [5]
    now.cuda_stream = 7                             # the current stream, without an argument
    calls[which]()
    assert plan.dev.seen == [5, 7]
    plan._own = False                               # a caller's buffer is the caller's
    calls[which](stream=Stream(9))
    assert plan.dev.seen == [5, 7]


@pytest.mark.parametrize("device", [None, "cuda", 0, "cuda:0"])
def test_a_plan_keeps_its_own_memory(device, monkeypatch):
    """Uploaded again, however the device is named: graphs captured over it and calls on other
    streams keep its address."""
    plan, _, _ = _uploaded(monkeypatch)
    mem = plan.dev
    mem.device, mem.is_cuda = torch.device("cuda:0"), True
    mem.get_device, mem.data_ptr, mem.copy_ = lambda: 0, lambda: 64, lambda *a, **k: None

    def other(*a, **k):
        raise AssertionError("allocated")

    monkeypatch.setattr(torch, "empty_like", other)
    plan.upload() if device is None else plan.upload(device)
    assert plan.dev is mem
    with pytest.raises(AssertionError, match="allocated"):
        plan.upload("cuda:1")


@pytest.mark.gpu
@pytest.mark.parametrize("args", [(), ("cuda",), (0,)])
def test_a_plans_address_after_more_uploads(args):
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    plan = bd.PagedPlan([1], [20], [[0, 1]], 4, 2, 64, page_size=16, num_pages=3)
    at = plan.upload(*args).dev.data_ptr()
    assert all(plan.upload(*args).dev.data_ptr() == at for _ in range(3))
    assert torch.equal(plan.dev.cpu(), torch.from_numpy(plan.host))


@pytest.mark.gpu
@pytest.mark.parametrize("ambient", [False, True])
def test_a_dropped_plan_is_read_to_the_end(ambient):
    """A plan dropped while its write waits on a side stream; other plans of the same size
    are uploaded at once."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    P, n = 16, 64
    pool = torch.zeros(2 * n, P, 2, 64, dtype=torch.bfloat16, device="cuda")
    cache = bd.PagedCache(pool, torch.zeros_like(pool))
    rows = torch.randn(n * P, 2, 64, device="cuda").bfloat16()
    lists = [np.random.default_rng(i).permutation(2 * n)[:n] for i in range(5)]

    def plan(i):
        return bd.PagedPlan([n * P], [n * P], [lists[i]], 4, 2, 64, page_size=P, num_pages=2 * n).upload()

    bd.bd_cache_write(plan(0), rows, rows, cache)   # first calls load the kernels
    pool.zero_()
    x = torch.randn(4096, 4096, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    p = plan(0)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):                         # some milliseconds in front of the write
            x = x @ x * 1e-3
    if ambient:
        with torch.cuda.stream(side):
            bd.bd_cache_write(p, rows, rows, cache)
    else:
        bd.bd_cache_write(p, rows, rows, cache, stream=side)
    at = p.dev.data_ptr()
    busy = not side.query()
    del p
    later = [plan(i) for i in range(1, 5)]
    assert not busy or all(q.dev.data_ptr() != at for q in later)
    torch.cuda.synchronize()
    assert busy, "the write was to wait"
    want = torch.zeros_like(pool)
    want[torch.from_numpy(lists[0]).cuda()] = rows.view(n, P, 2, 64)
    assert torch.equal(pool, want)


@pytest.mark.gpu
def test_capture_over_a_plans_own_memory():
    """Captured on another stream than the upload's, replayed while the plan is kept and other
    plans come and go."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    c = pu.Case([60, 1, 3], [2000, 700, 90], 8, 2, 128, page=32)
    want = pu.run_attention(c)
    q = c.q.cuda()
    out, lse = torch.empty_like(q), torch.empty(8, c.T, device="cuda")
    ws = torch.empty(bd.bd_paged_attn_workspace(c.plan), dtype=torch.uint8, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bd.bd_paged_attn(c.plan, q, c.cache, out, lse, ws)
    for _ in range(3):
        for _ in range(4):
            c.make_plan().upload()
        c.plan.upload()
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), want[0]) and torch.equal(lse.cpu(), want[1])

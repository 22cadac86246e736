"""Rotations used on other streams than the one they were made on."""
import pytest
import torch

bd = pytest.importorskip("block_causal_varlen_gb300")
paged = bd.paged


class Stream:
    def __init__(self, raw):
        self.cuda_stream = raw


class Memory:
    """Stands in for device memory: remembers which streams the allocator is told of."""

    def __init__(self):
        self.seen = []

    def record_stream(self, s):
        self.seen.append(s.cuda_stream)


def test_a_ropes_memory_is_known_to_be_used_on_other_streams(monkeypatch):
    rope = bd.Rope(torch.ones(32))
    plan = bd.PagedPlan([1], [20], [[0, 1]], 4, 2, 64, page_size=16, num_pages=3)
    plan.dev, plan._dev_ptr, plan._index = Memory(), 64, 0
    rope.phase, rope._index, rope._streams, now = Memory(), 0, {0}, Stream(0)    # as if made on raw stream 0 of device 0
    monkeypatch.setattr(paged, "_raw_stream", lambda i: now.cuda_stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: now)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(paged, "_device", lambda *a: 0)
    monkeypatch.setattr(paged, "_rows3", lambda *a: b"")
    monkeypatch.setattr(paged, "_entry", lambda n: lambda *a: 0)
    cache = bd.PagedCache(*(torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16) for _ in range(2)))

    def append(**k):
        bd.bd_cache_append(plan, None, None, None, rope, cache, **k)

    append()
    assert rope.phase.seen == []                    # the stream that it was made on
    append(stream=Stream(5))
    append(stream=Stream(5))
    assert rope.phase.seen == [5]
    now.cuda_stream = 7                             # the current stream, without an argument
    append()
    append()
    assert rope.phase.seen == [5, 7]


@pytest.mark.gpu
@pytest.mark.parametrize("ambient", [False, True])
def test_a_dropped_rope_is_read_to_the_end(ambient):
    """A rotation dropped while its append waits on a side stream; others of the same size are
    made at once."""
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    P, n, d = 16, 64, 128
    pools = [torch.zeros(n, P, 2, d, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    caches = [bd.PagedCache(x, torch.zeros_like(x)) for x in pools]
    rows = torch.randn(n * P, 2, d, device="cuda").bfloat16()
    plan = bd.PagedPlan([n * P], [n * P], [list(range(n))], 4, 2, d, page_size=P, num_pages=n).upload()

    def rope(i):
        return bd.Rope(torch.rand(d // 2, generator=torch.Generator().manual_seed(i)), device="cuda")

    bd.bd_cache_append(plan, None, rows, rows, rope(0), caches[0])
    x = torch.randn(4096, 4096, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    r = rope(0)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):                         # some milliseconds in front of the append
            x = x @ x * 1e-3
    if ambient:
        with torch.cuda.stream(side):
            bd.bd_cache_append(plan, None, rows, rows, r, caches[1])
    else:
        bd.bd_cache_append(plan, None, rows, rows, r, caches[1], stream=side)
    at = r.phase.data_ptr()
    busy = not side.query()
    del r
    later = [rope(i) for i in range(1, 5)]
    assert not busy or all(q.phase.data_ptr() != at for q in later)
    torch.cuda.synchronize()
    assert busy, "the append was to wait"
    assert torch.equal(pools[0], pools[1])

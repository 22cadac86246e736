"""Layouts that say nothing about a tensor: strides of dimensions of one element."""
import pytest
import torch

bd = pytest.importorskip("block_causal_varlen_gb300")
pu = pytest.importorskip("paged_util")
paged = bd.paged


def test_stride_of_a_single_row_of_lse(monkeypatch):
    """LSE of one new row as a view whose row stride is not 1."""
    plan = bd.PagedPlan([1], [20], [[0, 1]], 4, 2, 64, page_size=16, num_pages=3)
    sent = []
    monkeypatch.setattr(paged, "_device", lambda *a: -1)       # CPU tensors stand in
    monkeypatch.setattr(paged, "_rows3", lambda *a: b"")
    monkeypatch.setattr(paged, "_call", lambda fn, *a: sent.append(a))
    monkeypatch.setattr(paged, "_entry", lambda n: None)
    cache = bd.PagedCache(*(torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16) for _ in range(2)))
    ws = torch.empty(64, dtype=torch.uint8)
    bd.bd_paged_attn(plan, None, cache, None, torch.zeros(1, 4).t(), ws)
    bd.bd_paged_attn(plan, None, cache, None, torch.zeros(4, 7)[:, 3:4], ws)
    assert len(sent) == 2
    with pytest.raises(ValueError, match="lse"):
        bd.bd_paged_attn(plan, None, cache, None, torch.zeros(2, 4).t(), ws)


def test_strides_of_one_head_of_exponents():
    """One K/V head: the exponents' head stride has no meaning and need not agree."""
    pool = torch.zeros(3, 16, 1, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    ke = torch.zeros(3, 16, 1, dtype=torch.uint8)
    ve = torch.zeros(3, 1, 16, dtype=torch.uint8).transpose(1, 2)
    assert ke.stride() != ve.stride()
    bd.PagedCache(pool, pool, ke, ve)
    with pytest.raises(ValueError, match="strides"):
        bd.PagedCache(pool, pool, ke, torch.zeros(3, 32, 1, dtype=torch.uint8)[:, ::2])


@pytest.mark.gpu
def test_one_head_and_one_row():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    c = pu.Case([1], [300], 4, 1, 64, fmt="e4m3")
    want = pu.run_attention(c)
    P = c.page
    ve = c.ve.view(c.num_pages, 1, P).transpose(1, 2)
    c.cache = bd.PagedCache(c.k, c.v, c.ke, ve)
    lse = torch.full((1, 4), float("nan"), device="cuda").t()
    out = torch.empty(1, 4, 64, dtype=torch.bfloat16, device="cuda")
    bd.bd_paged_attn(c.plan, c.q.cuda(), c.cache, out, lse)
    assert torch.equal(out.cpu(), want[0]) and torch.equal(lse.cpu(), want[1])

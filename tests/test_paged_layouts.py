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

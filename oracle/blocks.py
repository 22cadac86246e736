"""Plain restatement of block bounds and block selection over a paged cache (test
infrastructure, CPU)."""
from __future__ import annotations

import math

import torch


def _power(top):
    """The smallest e of [-50, 50] with top <= 127 2^e (50 if there is none)."""
    e = -50
    while e < 50 and top > 127 * 2.0 ** e:
        e += 1
    return e


def bounds(k):
    """Keys k [n, d] of a block -> (lo codes, hi codes, exponent byte)."""
    k = k.double()
    if not torch.isfinite(k).all():
        z = torch.zeros(k.shape[1], dtype=torch.int8)
        return z, z.clone(), 255
    lo, hi = k.amin(0), k.amax(0)
    e = _power(max(lo.abs().max().item(), hi.abs().max().item()))
    f = 2.0 ** -e
    return (lo * f).floor().clamp(-127, 127).to(torch.int8), (hi * f).ceil().clamp(-127, 127).to(torch.int8), e + 127


def score(q, lo, hi, exp):
    """Score of a block for heads q [G, d]: exact, as a Python float."""
    if exp == 255:
        return math.inf
    best = -math.inf
    for row in q.double():
        ok = bool(torch.isfinite(row).all())
        e = _power(row.abs().max().item()) if ok else 0
        c = torch.round(row * 2.0 ** -e).clamp(-127, 127) if ok else torch.zeros_like(row)
        s = torch.maximum(c * lo.double(), c * hi.double()).sum().item()
        best = max(best, s * 2.0 ** (e + exp - 127))
    return best


def select(q, los, his, exps, blocks, first, recent):
    """The list of a row and K/V head: q [G, d], bounds of the blocks up to its own."""
    n = len(exps)
    if n <= blocks:
        return list(range(n)) + [-1] * (blocks - n)
    keep = set(range(first)) | set(range(n - recent, n))
    s = {j: score(q, los[j], his[j], int(exps[j])) for j in range(n) if j not in keep}
    order = sorted(s, key=lambda j: (-s[j], j))
    return sorted(keep | set(order[:blocks - len(keep)]))

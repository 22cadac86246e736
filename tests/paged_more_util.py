"""Helpers of the tests of 4-bit caches, rotated appends and selected blocks."""
from __future__ import annotations

import paged_util as pu
import torch

import block_causal_varlen_gb300 as bd
from oracle import paged as op
from oracle import paged_e2m1 as o4


class Case(pu.Case):
    """A batch over a random pool of any format. e2m1 pools: rows of different sizes; rows that
    nobody owns hold scales of NaN, unless `junk` is a number."""

    def __init__(self, new, kv, H, Hkv, d, page=16, fmt="bf16", heads_first=False, device="cuda", junk=float("nan"),
                 kmag=(-3, 2), vmag=(-6, 6), **kw):
        if fmt != "e2m1":
            super().__init__(new, kv, H, Hkv, d, page, fmt, heads_first, device=device, junk=junk, kmag=kmag, vmag=vmag, **kw)
            return
        super().__init__(new, kv, H, Hkv, d, page, "bf16", heads_first, device="cpu", junk=0.0, **kw)
        g = torch.Generator().manual_seed(kw.get("seed", 0) + 1000)
        shape, self.fmt = self.kd.shape, "e2m1"

        def place(t):
            t = t.to(device)
            return t.transpose(1, 2).contiguous().transpose(1, 2) if heads_first else t.contiguous()

        for n, mag in (("k", kmag), ("v", vmag)):
            x = getattr(self, n + "d") * 2.0 ** torch.randint(mag[0], mag[1] + 1, (*shape[:3], shape[3] // 16), generator=g).double().repeat_interleave(16, -1)
            x = x.bfloat16()
            x[~self.used] = junk
            c, s = o4.quantise(x)
            setattr(self, n + "d", o4.dequantise(c, s))
            setattr(self, n, place(c))
            setattr(self, n + "e", place(s))
        self.cache = bd.PagedCache(self.k, self.v, self.ke, self.ve)
        self.plan = self.make_plan()
        if device != "cpu":
            self.plan.upload(device)


def tolerances(d, keys, A, big, fmt, rows, vmax):
    """paged_util's bounds; for e2m1 with P as fp16 everywhere: rounded to 2^-11 of each, or (held
    times 2^7 and relative to a maximum that is 1 at least) 2^-32 absolute below 2^-21, times the largest
    |v| seen; the rest as for bf16. q is fp16 times a power of two: exact down to 2^-31 of the
    row's largest, which times the keys' sizes counts as the scores' own rounding does."""
    if fmt != "e2m1":
        return pu.tolerances(d, keys, A, big, fmt, rows)
    o, ls = pu.tolerances(d, keys, A, big, "bf16", rows)
    return o - A * (2.0 ** -8 - 2.0 ** -11) * 1.01 + keys * 2.0 ** -32 * vmax, ls


def check_attention(case, out, lse):
    """out, lse (CPU) against the oracle, every element."""
    at = 0
    for b, (n, kv) in enumerate(zip(case.new, case.kv)):
        if n:
            k, v = case.rows(b)
            o_ref, l_ref, A, big = op.attention(case.q[at:at + n], k, v, kv, case.causal)
            vmax = v.abs().max().item() if kv else 0.0
            to, tl = tolerances(case.d, max(kv, 1), A, big, case.fmt, n * case.H // case.Hkv, vmax)
            compare(out[at:at + n], lse[:, at:at + n], o_ref, l_ref, to, tl, (b, n, kv))
        at += n


def compare(out, lse, o_ref, l_ref, to, tl, what):
    got, gl = out.double(), lse.double()
    empty = torch.isneginf(l_ref)
    assert torch.equal(torch.isneginf(gl), empty), (what, "rows that see nothing")
    if empty.any():
        assert (got.permute(1, 0, 2)[empty] == 0).all(), (what, "O of rows that see nothing")
    assert torch.isfinite(got).all(), (what, "O not finite")
    bad = (got - o_ref).abs() > to
    assert not bad.any(), (what, bad.sum().item(), (got - o_ref).abs().max().item(), bad.nonzero()[:4].tolist())
    bad = ((gl - l_ref).abs() > tl) & ~empty
    assert not bad.any(), (what, "LSE", (gl - l_ref)[~empty].abs().max().item())

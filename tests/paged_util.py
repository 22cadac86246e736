"""Helpers of the paged-cache tests: pools, plans, the oracle's outputs and the
tolerances, which follow from the roundings the kernels make."""
from __future__ import annotations

import numpy as np
import torch

import block_causal_varlen_gb300 as bd
from oracle import paged as op


class Case:
    """A batch over a random pool. `new` / `kv`: new rows and cached rows of every
    sequence. Rows of the pool nobody owns, and rows past kv_len of a last page, hold
    NaN unless `junk` says otherwise."""

    def __init__(self, new, kv, H, Hkv, d, page=16, fmt="bf16", heads_first=False, causal=True, seed=0, spare=2,
                 device="cuda", junk=float("nan"), qscale=1.0, pad_rows=0, kmag=(-3, 2),
                 vmag=(-6, 6)):
        g = torch.Generator().manual_seed(seed)
        self.new, self.kv, self.H, self.Hkv, self.d, self.page = list(new), list(kv), H, Hkv, d, page
        self.fmt, self.causal = fmt, causal
        n_pages = [-(-n // page) for n in kv]
        self.num_pages = sum(n_pages) + spare
        order = np.random.default_rng(seed).permutation(self.num_pages)
        cut = np.cumsum([0] + n_pages)
        self.pages = [order[cut[b]:cut[b + 1]].tolist() for b in range(len(kv))]
        shape = (self.num_pages, page, Hkv, d)
        k, v = torch.randn(shape, generator=g), torch.randn(shape, generator=g)
        if fmt == "e4m3":  # rows of different sizes
            k = k * 2.0 ** torch.randint(kmag[0], kmag[1] + 1, shape[:3], generator=g)[..., None]
            v = v * 2.0 ** torch.randint(vmag[0], vmag[1] + 1, shape[:3], generator=g)[..., None]
        used = torch.zeros(self.num_pages, page, dtype=torch.bool)
        for n, pg in zip(kv, self.pages):
            for j in range(0, n, page):
                used[pg[j // page], :min(page, n - j)] = True
        k, v = k.bfloat16(), v.bfloat16()
        k[~used] = junk
        v[~used] = junk
        self.used = used
        T = sum(new)
        self.T = T
        self.q = (torch.randn(T + pad_rows, H, d, generator=g) * qscale).bfloat16()
        self.k_new = torch.randn(T + pad_rows, Hkv, d, generator=g).bfloat16()
        self.v_new = torch.randn(T + pad_rows, Hkv, d, generator=g).bfloat16()

        def place(t):  # the pool in either order of its dimensions, as [page, row, head, ...]
            t = t.to(device)
            if not heads_first:
                return t.contiguous()
            dims = (0, 2, 1, 3)[:t.dim()]
            return t.permute(dims).contiguous().permute(dims)

        if fmt == "e4m3":
            (kc, ke), (vc, ve) = op.quantise(k), op.quantise(v)
            self.kd, self.vd = op.dequantise(kc, ke), op.dequantise(vc, ve)
            self.k, self.v = place(kc).view(torch.float8_e4m3fn), place(vc).view(torch.float8_e4m3fn)
            self.ke, self.ve = place(ke), place(ve)
        else:
            self.kd, self.vd = k.double(), v.double()
            self.k, self.v, self.ke, self.ve = place(k), place(v), None, None
        self.cache = bd.PagedCache(self.k, self.v, self.ke, self.ve)
        self.plan = self.make_plan()
        if device != "cpu":
            self.plan.upload(device)

    def make_plan(self, **kw):
        a = dict(q_len=self.new, kv_len=self.kv, pages=self.pages, H=self.H, Hkv=self.Hkv, d=self.d, page_size=self.page,
                 num_pages=self.num_pages, fmt=self.cache.fmt, causal=self.causal)
        a.update(kw)
        return bd.PagedPlan(**a)

    def rows(self, b):
        return (op.rows_of(self.kd, self.kv[b], self.pages[b], self.page),
                op.rows_of(self.vd, self.kv[b], self.pages[b], self.page))


def tolerances(d, keys, A, big, fmt, rows=1):
    """(O, LSE) bounds. A = sum p |v| per output, big = max_j sum |q k_j| / sqrt(d) per row.
    Score: products of the operands are exact in fp32, their sum of d terms is off by at
    most d 2^-24 of the sum of magnitudes (twice that allows for chopped additions), the
    factor log2(e) / sqrt(d), the exponent's base change and the subtraction of m by
    2^-22 of the same: ds = (2 d + 8) 2^-24 big, plus 2^-22 for the exponential itself.
    l: a sum of `keys` terms in parts: keys 2^-24 relative at most; the logarithm 2^-21
    absolute and its rounding 2^-23 of |LSE| (< 64 here: 2^-17).
    O: P rounded to half a step (2^-11 of each term where it is fp16: e4m3 caches, `rows`
    (new row, head) pairs of a K/V head up to 16, i.e. the few-rows kernel; 2^-8 where it
    is bf16, i.e. bf16 caches and the tile kernel, whose e4m3 tiles are bf16 by then),
    which sum to at most that times A, products summed as above, and the output rounded by
    2^-8 of itself (applied to A, which is no smaller). Few-rows e4m3 blocks (up to 48 pairs)
    hold p 2^e (e: V's exponent) as fp16, the largest of a row at 2^7 at least: below 2^-14
    its rounding is 2^-25 absolute, 2^-32 of the largest, times a code of at most 448. The
    key with the largest has a code above 224 somewhere (its row's maximum), where A is at
    least 224 times it: the sum over the keys is within keys 2^-31 of A's largest column.
    (It counts where the keys with the largest p have zeros in a column.)"""
    ds = (2 * d + 8) * 2.0 ** -24 * big + 2.0 ** -22
    ls = ds + keys * 2.0 ** -24 + 2.0 ** -21 + 2.0 ** -17
    p = 2.0 ** -11 if fmt == "e4m3" and rows <= 16 else 2.0 ** -8
    o = A * (p + 2.0 ** -8) * 1.01 + A * (2 * ls.t()[..., None] + 2 * keys * 2.0 ** -24) + 1e-30
    if fmt == "e4m3" and rows <= 48:
        o = o + keys * 2.0 ** -31 * A.amax(-1, keepdim=True)
    return o, ls


def check_attention(case, out, lse):
    """out, lse (CPU) against the oracle, every element."""
    at = 0
    for b, (n, kv) in enumerate(zip(case.new, case.kv)):
        if n:
            k, v = case.rows(b)
            o_ref, l_ref, A, big = op.attention(case.q[at:at + n], k, v, kv, case.causal)
            tol_o, tol_l = tolerances(case.d, max(kv, 1), A, big, case.fmt, n * case.H // case.Hkv)
            got, gl = out[at:at + n].double(), lse[:, at:at + n].double()
            empty = torch.isneginf(l_ref)
            assert torch.equal(torch.isneginf(gl), empty), f"sequence {b}: rows that see nothing"
            if empty.any():
                assert (got.permute(1, 0, 2)[empty] == 0).all(), f"sequence {b}: O of rows that see nothing"
            assert torch.isfinite(got).all(), f"sequence {b}: O not finite"
            bad = (got - o_ref).abs() > tol_o
            assert not bad.any(), (b, n, kv, bad.sum().item(), (got - o_ref).abs().max().item(), bad.nonzero()[:4].tolist())
            bad = ((gl - l_ref).abs() > tol_l) & ~empty
            assert not bad.any(), (b, n, kv, "LSE", (gl - l_ref)[~empty].abs().max().item())
        at += n


def run_attention(case, stream=None, poison=True, workspace=None):
    out = torch.full((case.q.shape[0], case.H, case.d), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((case.H, case.q.shape[0]), float("nan"), device="cuda")
    if workspace is None:
        workspace = torch.full((max(1, bd.bd_paged_attn_workspace(case.plan)),), 255, dtype=torch.uint8, device="cuda")
    bd.bd_paged_attn(case.plan, case.q.cuda(), case.cache, out, lse, workspace, stream=stream)
    torch.cuda.synchronize()
    bd.bd_check_status(case.plan)
    return out.cpu(), lse.cpu()

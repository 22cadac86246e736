"""Plain float64 restatement of the paged K/V cache (test infrastructure, CPU): the
e4m3 row format, where new rows go, and attention of new rows over cached ones."""
from __future__ import annotations

import math

import torch

# magnitudes of the e4m3 codes 0x00..0x7e: 3 mantissa bits, exponent bias 7, no infinities
E4M3 = torch.tensor([(m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                     for e in range(16) for m in range(8)][:127], dtype=torch.float64)


def decode_e4m3(codes):
    """Values of uint8 codes."""
    c = codes.long()
    mag = torch.cat([E4M3, torch.tensor([math.nan], dtype=torch.float64)])[c & 127]
    return torch.where(c >= 128, -mag, mag)


def quantise(x):
    """(codes, exponent bytes) of rows x [..., d]: per row the smallest e in [-60, 60]
    with max|x| <= 448 2^e, each code the nearest of all codes to x 2^-e (ties to the
    even one); a row with an infinity or a NaN is NaN codes and byte 255."""
    x = x.double()
    bad = ~torch.isfinite(x).all(-1)
    y = torch.where(bad[..., None], torch.zeros_like(x), x)
    top = y.abs().amax(-1)
    e = torch.full(top.shape, -60, dtype=torch.long)
    for k in range(-60, 60):
        e = torch.where(top > 448.0 * 2.0 ** k, k + 1, e)
    a = y.abs() * 2.0 ** (-e.double())[..., None]
    hi = torch.searchsorted(E4M3, a.contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    dh, dl = E4M3[hi] - a, a - E4M3[lo]
    code = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = torch.where(a >= 448.0, 126, code)
    code = code + 128 * torch.signbit(y).long()
    code = torch.where(bad[..., None], 127, code)
    return code.to(torch.uint8), torch.where(bad, 255, e + 127).to(torch.uint8)


def dequantise(codes, exps):
    """Values of codes [..., d] and exponent bytes [...]; byte 255 gives NaN."""
    f = 2.0 ** (exps.double() - 127)
    f = torch.where(exps.long() == 255, math.nan, f)
    return decode_e4m3(codes) * f[..., None]


def slots(q_len, kv_len, pages, page_size):
    """Cache row (page * page_size + row) of every packed new row, -1 for none."""
    out = []
    for q, n, pg in zip(q_len, kv_len, pages):
        for i in range(q):
            pos = n - q + i
            out.append(-1 if pos < 0 else int(pg[pos // page_size]) * page_size + pos % page_size)
    return out


def rows_of(pool, n, pages, page_size):
    """Rows [0, n) of a sequence from a pool [pages, page_size, ...]."""
    return torch.stack([pool[int(pages[j // page_size]), j % page_size] for j in range(n)]) if n else pool[:0, 0]


def attention(q, k, v, kv_len, causal=True):
    """q [nq, H, d], k, v [kv_len, Hkv, d] -> O [nq, H, d], LSE [H, nq], and two sizes
    tolerances are made of: sum_j p_j |v_j| per output, max_j sum |q_i k_ji| / sqrt(d)
    per row."""
    nq, H, d = q.shape
    G = H // k.shape[1]
    q, k, v = q.double(), k.double().repeat_interleave(G, 1), v.double().repeat_interleave(G, 1)
    if kv_len == 0:
        z = torch.zeros(nq, H, d, dtype=torch.float64)
        return z, torch.full((H, nq), -math.inf, dtype=torch.float64), z, torch.zeros(H, nq, dtype=torch.float64)
    s = torch.einsum("ihd,jhd->hij", q, k) / math.sqrt(d)
    big = torch.einsum("ihd,jhd->hij", q.abs(), k.abs()) / math.sqrt(d)
    if causal:
        i, j = torch.arange(nq)[:, None], torch.arange(kv_len)[None]
        hide = j > kv_len - nq + i
        s = s.masked_fill(hide, -math.inf)
        big = big.masked_fill(hide, 0.0)
    m = s.amax(-1, keepdim=True)
    m = torch.where(torch.isneginf(m), torch.zeros_like(m), m)
    p = torch.exp(s - m)
    tot = p.sum(-1, keepdim=True)
    lse = (m + torch.log(tot))[..., 0]
    p = p / torch.where(tot == 0, torch.ones_like(tot), tot)
    return torch.einsum("hij,jhd->ihd", p, v), lse, torch.einsum("hij,jhd->ihd", p, v.abs()), big.amax(-1)

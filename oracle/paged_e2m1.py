"""Plain float64 restatement of the e2m1 format of a paged K/V cache (test infrastructure, CPU)."""
from __future__ import annotations

import math

import torch

# magnitudes of the codes 0..7, and the scales of the bytes 0..226 (3 mantissa bits, bias 15)
E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
SCALES = torch.tensor([m / 8 * 2.0 ** -14 if e == 0 else (1 + m / 8) * 2.0 ** (e - 15)
                       for e in range(32) for m in range(8)][:227], dtype=torch.float64)


def scales_of(bytes_):
    """Values of scale bytes; those past 226 are NaN."""
    return torch.cat([SCALES, torch.full((29,), math.nan, dtype=torch.float64)])[bytes_.long()]


def quantise(x):
    """(packed codes [..., d / 2], scale bytes [..., d / 16]) of rows x [..., d]: for every 16
    values the smallest byte of [8, 226] with max|x| <= 6 s, each code the nearest of all codes to
    x / s (ties to the even one); 16 values with an infinity or a NaN are byte 255 and zeros."""
    g = x.double().unflatten(-1, (-1, 16))
    bad = ~torch.isfinite(g).all(-1)
    g = torch.where(bad[..., None], torch.zeros_like(g), g)
    top = g.abs().amax(-1)
    byte = torch.full(top.shape, 8, dtype=torch.long)
    for b in range(8, 226):
        byte = torch.where(top > 6 * SCALES[b], b + 1, byte)
    y = g.abs() / SCALES[byte][..., None]
    code = torch.zeros_like(y, dtype=torch.long)
    for c in range(7):
        mid = (E2M1[c] + E2M1[c + 1]) / 2
        code = torch.where((y > mid) | ((y == mid) & ((c + 1) % 2 == 0)), c + 1, code)
    code = torch.where(bad[..., None], 0, code + 8 * torch.signbit(g).long()).flatten(-2)
    return (code[..., 0::2] + 16 * code[..., 1::2]).to(torch.uint8), torch.where(bad, 255, byte).to(torch.uint8)


def dequantise(codes, scales):
    """Values of packed codes [..., d / 2] and scale bytes [..., d / 16]."""
    both = torch.cat([E2M1, -E2M1])
    c = codes.long()
    x = torch.stack([both[c & 15], both[c >> 4]], -1).flatten(-2)
    return (x.unflatten(-1, (-1, 16)) * scales_of(scales)[..., None]).flatten(-2)

"""Plain restatement of a position rotation (test infrastructure, CPU): angles reduced in exact
arithmetic, turned in float64."""
from __future__ import annotations

import math
from fractions import Fraction

import torch

_PI = Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534211706798")


def angles(positions, inv_freq):
    """Angles [len(positions), len(inv_freq)] in (-pi, pi], from exact products."""
    out = []
    for p in positions:
        row = []
        for f in inv_freq:
            turns = Fraction(float(f)) * int(p) / (2 * _PI)
            turns -= round(turns)
            row.append(float(turns * 2 * _PI))
        out.append(row)
    return torch.tensor(out, dtype=torch.float64).reshape(len(out), len(inv_freq))


def turn(x, positions, inv_freq, interleaved=False, scale=1.0):
    """Rows x [T, heads, d] turned by their positions, float64; rows of negative position as they are."""
    r = 2 * len(inv_freq)
    a = angles([max(0, int(p)) for p in positions], inv_freq)[:, None]
    y = x.double().clone()
    i, j = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    u, v = x.double()[..., i], x.double()[..., j]
    y[..., i], y[..., j] = scale * (u * a.cos() - v * a.sin()), scale * (v * a.cos() + u * a.sin())
    there = torch.tensor([int(p) >= 0 for p in positions])[:, None, None]
    return torch.where(there, y, x.double())


def lengths(x, inv_freq, interleaved=False):
    """Length of every element's pair (1-norm), float64; 0 for elements that stay."""
    r = 2 * len(inv_freq)
    y = torch.zeros_like(x, dtype=torch.float64)
    i, j = (slice(0, r, 2), slice(1, r, 2)) if interleaved else (slice(0, r // 2), slice(r // 2, r))
    n = x.double()[..., i].abs() + x.double()[..., j].abs()
    y[..., i], y[..., j] = n, n
    return y


assert math.isclose(float(_PI), math.pi)

"""Norms per head and rotary positions in 64 bits on the CPU, for the tests of the operators that apply them.

norm_rotate is the definition:
    y = x w / sqrt(mean(x^2) + eps)  (w None: y = x),  the pairs (a, b) -> (a c - b s, a s + b c),
    c = amplitude cos(p f_i), s = amplitude sin(p f_i)
Angles of far positions are reduced in whole numbers, since p f_i in 64 bits is off by p f_i 2^-53.
"""
import math
from fractions import Fraction

import torch

EPS = 1e-6
# pi to 400 bits, by Machin's formula
_ONE = 1 << 400


def _arctan_inverse(x):
    t = s = _ONE // x
    n, sign = 1, -1
    while t:
        t //= x * x
        n += 2
        s += sign * (t // n)
        sign = -sign
    return s


_TWO_PI = Fraction(2 * 4 * (4 * _arctan_inverse(5) - _arctan_inverse(239)), _ONE)


def angles(positions, freq):
    """p f modulo a turn, within [0, 2 pi), in 64 bits: [*positions.shape, len(freq)]."""
    rows = []
    for f in freq.tolist():
        turn = Fraction(f) / _TWO_PI
        rows.append([float((p * turn) % 1) * 2 * math.pi for p in positions.reshape(-1).tolist()])
    return torch.tensor(rows, dtype=torch.float64).reshape(len(rows), -1).T.reshape(*positions.shape, len(rows))


def positions(B, N, start=None, offsets=None):
    p = torch.arange(N).expand(B, N) if offsets is None else offsets.long().expand(B, N)
    return p if start is None else p + start.long()[:, None]


def _pairs(rot, layout):
    if layout == "half":
        return slice(0, rot // 2), slice(rot // 2, rot)
    return slice(0, rot, 2), slice(1, rot, 2)


def _inverse_rms(x, eps):
    return 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)


def norm_rotate(x, freq, pos, layout="half", amplitude=1.0, weight=None, eps=EPS):
    """(y, size) of x [B, H, N, d] at pos [B, N]: the result in 64 bits, and for each component what its error counts in."""
    y = x.double()
    if weight is not None:
        y = y * _inverse_rms(y, eps) * weight.double()
    size = y.abs()
    if freq is not None and len(freq):
        rot = 2 * len(freq)
        t = angles(pos, freq)[:, None]
        c, s = amplitude * t.cos(), amplitude * t.sin()
        a, b = _pairs(rot, layout)
        out, size = y.clone(), size.clone()
        out[..., a] = y[..., a] * c - y[..., b] * s
        out[..., b] = y[..., a] * s + y[..., b] * c
        size[..., a] = size[..., b] = abs(amplitude) * (y[..., a].abs() + y[..., b].abs())
        y = out
    return y, size


def gradients(dy, x, freq, pos, layout="half", amplitude=1.0, weight=None, eps=EPS):
    """(dx, dw, size of dx, size of dw) of norm_rotate, in 64 bits."""
    g, size = norm_rotate(dy, None if freq is None else -freq, pos, layout, amplitude)
    if weight is None:
        return g, None, size, None
    x = x.double()
    r = _inverse_rms(x, eps)
    xr, w = x * r, weight.double()
    dw = (g * xr).sum((0, 1, 2))
    dx = r * (g * w - xr * (g * w * xr).mean(-1, keepdim=True))
    weighted = size * w.abs()
    return dx, dw, r * (weighted + xr.abs() * (weighted * xr.abs()).mean(-1, keepdim=True)), (size * xr.abs()).sum((0, 1, 2))

"""Oracle of the rotary positions: numpy in 64 bits, frequencies as exact fractions."""
from __future__ import annotations

from fractions import Fraction

import numpy as np

TWO_PI = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459")


def turns(inv_freq):
    """Turns a position in units of 2^-64, modulo 2^64, as signed whole numbers."""
    out = []
    for f in inv_freq:
        w = round(Fraction(float(f)) * 2 ** 64 / TWO_PI) % 2 ** 64
        out.append(w - 2 ** 64 if w >= 2 ** 63 else w)
    return out


def angles(positions, turn_units, pair_axis=None):
    """Angles [T, pairs] of positions [axes, T]: the fraction of a turn by whole numbers."""
    pos = [[int(p) for p in axis] for axis in positions]
    pairs = len(turn_units)
    axis = list(pair_axis) if pair_axis is not None else [0] * pairs
    out = np.empty((len(pos[0]), pairs))
    for t in range(len(pos[0])):
        for i in range(pairs):
            part = pos[axis[i]][t] * int(turn_units[i]) % 2 ** 64
            out[t, i] = float(Fraction(part - 2 ** 64 if part >= 2 ** 63 else part, 2 ** 64)
                              * TWO_PI)
    return out


def pairs_of(rotary, interleaved):
    """The elements of each pair, as two index arrays."""
    i = np.arange(rotary // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rotary // 2)


def rope(x, angle, interleaved=False, inverse=False, magnitude=1.0):
    """x [T, H, D] (anything numpy takes) rotated by angle [T, pairs], in float64."""
    x = np.asarray(x, dtype=np.float64)
    a, b = pairs_of(2 * angle.shape[1], interleaved)
    c = np.cos(angle)[:, None] * magnitude
    s = np.sin(angle)[:, None] * magnitude * (-1 if inverse else 1)
    out = x.copy()
    out[..., a] = x[..., a] * c - x[..., b] * s
    out[..., b] = x[..., b] * c + x[..., a] * s
    return out

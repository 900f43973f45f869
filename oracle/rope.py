"""Oracle of the rotary positions (numpy, extended precision): frequencies, rotation, gradient.

Parity status (pins live in tests/test_oracle_rope.py): complex rotation by hand, inverse of
itself, dot products that depend on the distance alone, differences for the gradient.
"""
from __future__ import annotations

import math

import numpy as np


def freqs(rot, base=10000.0, scaling="none", factor=1.0, trained=0.0, low=1.0, high=32.0):
    """Radians per position, fp64 [rot / 2]."""
    out = np.empty(rot // 2)
    for i in range(rot // 2):
        b = base * factor ** (rot / (rot - 2)) if scaling == "base" else base
        w = b ** (-2.0 * i / rot)
        if scaling == "linear":
            w /= factor
        if scaling == "ramp":
            turns = trained * w / (2 * math.pi)
            c = min(1.0, max(0.0, (turns - low) / (high - low)))
            w = c * w + (1 - c) * w / factor
        out[i] = w
    return out


def positions(n, cu, start=None):
    """Position of each row of a packed batch, None behind the last sequence."""
    out = [None] * n
    for s in range(len(cu) - 1):
        for t in range(int(cu[s]), min(int(cu[s + 1]), n)):
            out[t] = (0 if start is None else int(start[s])) + t - int(cu[s])
    return out


def rotate(x, pos, w, interleaved, mscale=1.0, sign=1):
    """x [n, h, d] turned by sign times its positions; rows of position None stay."""
    x = np.asarray(x, np.float64)
    y, half = x.copy(), len(w)
    a = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    b = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    for t, p in enumerate(pos):
        if p is None:
            continue
        angle = np.longdouble(p) * w.astype(np.longdouble)
        c = (np.cos(angle) * mscale).astype(np.float64)
        s = (np.sin(angle) * mscale * sign).astype(np.float64)
        y[t, :, a] = x[t, :, a] * c - x[t, :, b] * s
        y[t, :, b] = x[t, :, b] * c + x[t, :, a] * s
    return y

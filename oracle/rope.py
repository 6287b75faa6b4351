"""Rotary positions in float64.

Test infrastructure only (see ``oracle/__init__``).

Pair j of a head's rotated part turns by p * f_j at position p:
(a, b) -> (a cos - b sin, b cos + a sin).  ``frequencies`` states f_j for
each scaling; positions and frequencies are float64 (p < 2^31, f_j <= 1: the
angle is off by 2^31 * 2^-53 = 2^-22 radians at most, at the largest positions).
"""

import math

import numpy as np


def frequencies(rot, theta=10000.0, scaling="none", factor=1.0, original=0, low=0.0, high=0.0):
    if scaling == "ntk":
        theta = theta * factor ** (rot / (rot - 2))
    out = []
    if scaling == "yarn":
        first = max(math.floor(rot * math.log(original / (high * 2 * math.pi)) / (2 * math.log(theta))), 0)
        last = min(math.ceil(rot * math.log(original / (low * 2 * math.pi)) / (2 * math.log(theta))), rot - 1)
        if last <= first:
            last = first + 0.001
    for j in range(rot // 2):
        f = theta ** (-2.0 * j / rot)
        if scaling == "linear":
            f = f / factor
        elif scaling == "yarn":
            w = min(max((j - first) / (last - first), 0.0), 1.0)
            f = f / factor * w + f * (1 - w)
        elif scaling == "banded":
            w = min(max((original * f / (2 * math.pi) - low) / (high - low), 0.0), 1.0)
            f = f / factor * (1 - w) + f * w
        out.append(f)
    return np.array(out)


def rotate(x, positions, freq, offset=0, pairs=False, amplitude=1.0):
    """x [n, heads, d] float64 with the 2 len(freq) elements from ``offset`` turned by each row's position."""
    x = np.asarray(x, dtype=np.float64)
    y = x.copy()
    t = np.asarray(positions, dtype=np.float64)[:, None, None] * np.asarray(freq)
    c, s = amplitude * np.cos(t), amplitude * np.sin(t)
    h = len(freq)
    if pairs:
        ia, ib = slice(offset, offset + 2 * h, 2), slice(offset + 1, offset + 2 * h, 2)
    else:
        ia, ib = slice(offset, offset + h), slice(offset + h, offset + 2 * h)
    a, b = x[..., ia], x[..., ib]
    y[..., ia] = a * c - b * s
    y[..., ib] = b * c + a * s
    return y

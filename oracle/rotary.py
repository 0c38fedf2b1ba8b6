"""Rotary positions, written out plainly in numpy (test oracle).

Pair i of a head, at position p, turns by p * theta_i; angles are taken from the
64-bit fractions of a turn in whole-number arithmetic, so they are exact, and
everything else is fp64.  Test infrastructure only.
"""
from __future__ import annotations

import math

import numpy as np


def thetas(rot, scaling="plain", base=10000.0, factor=1.0, context=0.0, low=1.0, high=32.0):
    """Angle a position adds to each pair, one by one, and the scale of cosines and sines."""
    out, scale = [], 1.0
    for i in range(rot // 2):
        b = base * factor ** (rot / (rot - 2)) if scaling == "base" else base
        t = math.exp(-2.0 * i / rot * math.log(b))
        if scaling == "linear":
            t /= factor
        elif scaling == "bands":
            turns = context * t / (2 * math.pi)
            if turns <= low:
                t = t / factor
            elif turns < high:
                share = (turns - low) / (high - low)
                t = share * t + (1 - share) * t / factor
        elif scaling == "ramp":
            def number(turns):
                return rot * math.log(context / (turns * 2 * math.pi)) / (2 * math.log(base))
            a, z = max(0, math.floor(number(high))), min(rot - 1, math.ceil(number(low)))
            share = min(1.0, max(0.0, (i - a) / max(z - a, 0.001)))
            t = (1 - share) * t + share * t / factor
            scale = 0.1 * math.log(factor) + 1
        out.append(t)
    return np.array(out), scale


def angles(pos, turns):
    """[rows][pairs] angles of whole positions, from the 64 bits of the turns."""
    out = np.empty((len(pos), len(turns)))
    for r, p in enumerate(pos):
        for i, t in enumerate(turns):
            out[r, i] = ((int(p) * int(t)) % (1 << 64)) / 2.0 ** 64 * (2 * math.pi)
    return out


def rotate(x, pos, heads, rot, layout, turns, scale):
    """Rows x [n][heads*d] rotated, fp64, and what an fp32 evaluation (cosine and sine rounded, three roundings a value)
    may be off, before the result is rounded to its type."""
    n, d = x.shape[0], x.shape[1] // heads
    y = np.asarray(x, np.float64).reshape(n, heads, d).copy()
    tol = np.zeros_like(y)
    ang = angles(pos, turns)
    for i in range(rot // 2):
        a, b = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
        c, s = scale * np.cos(ang[:, i])[:, None], scale * np.sin(ang[:, i])[:, None]
        u, v = y[:, :, a].copy(), y[:, :, b].copy()
        y[:, :, a], y[:, :, b] = u * c - v * s, u * s + v * c
        size = np.abs(u) * abs(scale) + np.abs(v) * abs(scale)
        # c and s to half a step of fp32 (and 2^-35 in all), their products, and the sum
        tol[:, :, a] = tol[:, :, b] = (3 * 2.0 ** -24 + 2.0 ** -34) * size + 2.0 ** -148
    return y.reshape(n, -1), tol.reshape(n, -1)

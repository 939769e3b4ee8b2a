"""Packed-row operators, plainly, in float64: the norm with the residual's
addition, the gated activation, rows in eight bits, the projection of such
rows, and the rotary map with its scalings."""
from __future__ import annotations

import math

import numpy as np

TINY = 2.0 ** -126


def norm(x, weight, eps, residual=None):
    """(h, y): the sum and its norm times the weights, rows in the first axis."""
    h = x if residual is None else x + residual
    return h, h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * weight


def swiglu(gate_up):
    g, u = np.split(gate_up, 2, -1)
    with np.errstate(over="ignore"):
        return g / (1 + np.exp(-g)) * u


def scales(y):
    """One scale a row: the largest magnitude over 127; 0 below 2^-126, NaN where the row is not finite."""
    with np.errstate(invalid="ignore"):
        s = np.abs(y).max(-1) / 127
    return np.where(np.isfinite(s), np.where(s < TINY, 0, s), np.nan)


def linear(codes, row_scale, w_codes, w_scale, bias=None):
    """Integer sums, times both scales, plus the bias."""
    acc = codes.astype(np.int64) @ w_codes.astype(np.int64).T
    y = acc * row_scale[:, None] * w_scale
    return y if bias is None else y + bias


# ---------------------------------------------------------------- rotary map
def frequencies(rot, scaling="plain", theta=10000.0, factor=1.0, low=0.0, high=0.0, original_len=0):
    """(radians a position of each pair, factor of cos and sin)."""
    f = np.array([theta ** (-2.0 * i / rot) for i in range(rot // 2)])
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "ntk":
        return np.array([(theta * factor ** (rot / (rot - 2))) ** (-2.0 * i / rot) for i in range(rot // 2)]), 1.0
    if scaling == "bands":
        out = []
        for x in f:
            turns = original_len / (2 * math.pi / x)   # wavelengths the trained length holds
            if turns >= high:
                out.append(x)
            elif turns <= low:
                out.append(x / factor)
            else:
                w = (turns - low) / (high - low)
                out.append(w * x + (1 - w) * x / factor)
        return np.array(out), 1.0
    if scaling == "yarn":
        def pair(turns):
            return rot * math.log(original_len / (turns * 2 * math.pi)) / (2 * math.log(theta))
        a, b = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), rot - 1)
        out = []
        for i, x in enumerate(f):
            r = min(1.0, max(0.0, (i - a) / (b - a if b > a else 1e-3)))
            out.append(x / factor * r + x * (1 - r))
        return np.array(out), 0.1 * math.log(factor) + 1.0
    return f, 1.0


def rotate(x, positions, turns, attn=1.0, layout="half", inverse=False):
    """Heads x [n, heads, dh] turned at integer positions [n]; turns: the
    fractions of a turn a position of each pair, times 2^64, as Python
    integers, so that no angle is rounded before it is reduced."""
    half = len(turns)
    out = np.array(x, np.float64)
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if layout == "interleaved" else (i, i + half)
    for r, g in enumerate(positions):
        part = np.array([(int(g) * int(t)) % (1 << 64) for t in turns], np.float64) / 2.0 ** 64
        c, s = np.cos(2 * np.pi * part), np.sin(2 * np.pi * part)
        m = 1 / attn if inverse else attn
        c, s = c * m, (-s if inverse else s) * m
        u, w = x[r][:, a].astype(np.float64), x[r][:, b].astype(np.float64)
        out[r][:, a], out[r][:, b] = u * c - w * s, w * c + u * s
    return out

"""Paged cache, plainly: rows in and out of pages and attention over them.

The 4-bit rows and the rotation are defined in fp32 (each product and sum
rounded on its own), so append() is evaluated in float32 and its bits are the
definition; attention is float64."""
from __future__ import annotations

import numpy as np


def rope_table(n: int, dh: int, theta: float) -> np.ndarray:
    """fp32 (cos, sin) [n, dh/2, 2], the angles formed in float64."""
    a = np.arange(n)[:, None] * theta ** (-2.0 * np.arange(dh // 2) / dh)
    return np.stack([np.cos(a), np.sin(a)], -1).astype(np.float32)


def rotate(x: np.ndarray, cs: np.ndarray) -> np.ndarray:
    """Rotate-half of fp32 rows [n, heads, dh] by cs [n, dh/2, 2], in fp32."""
    h = x.shape[-1] // 2
    a, b = x[..., :h], x[..., h:]
    c, s = cs[:, None, :, 0], cs[:, None, :, 1]
    return np.concatenate([a * c - b * s, b * c + a * s], -1)


def quantise(x: np.ndarray, group: int):
    """Codes uint8 [..., dh] and fp16 (scale, offset) [..., dh/group, 2] of fp32 x."""
    g = np.clip(x, np.float32(-32768), np.float32(32768)).reshape(*x.shape[:-1], -1, group)
    lo, hi = g.min(-1), g.max(-1)
    s = ((hi - lo) * np.float32(1.0 / 15.0)).astype(np.float16)
    o = lo.astype(np.float16)
    sf = s.astype(np.float32)
    inv = np.where(sf > 0, np.float32(1) / np.where(sf > 0, sf, np.float32(1)), np.float32(0))
    code = np.clip(np.rint((g - o.astype(np.float32)[..., None]) * inv[..., None]), 0, 15)
    return code.astype(np.uint8).reshape(x.shape), np.stack([s, o], -1)


def pack(code: np.ndarray) -> np.ndarray:
    """Codes [..., 128] to the stored 64 bytes: unit u (dims 4u..4u+3, low
    nibble first) at two-byte place 4 (u % 8) + u // 8."""
    out = np.zeros((*code.shape[:-1], 64), np.uint8)
    for u in range(32):
        place = 4 * (u % 8) + u // 8
        c = code[..., 4 * u:4 * u + 4]
        out[..., 2 * place] = c[..., 0] | (c[..., 1] << 4)
        out[..., 2 * place + 1] = c[..., 2] | (c[..., 3] << 4)
    return out


def unpack(rows: np.ndarray) -> np.ndarray:
    code = np.zeros((*rows.shape[:-1], 128), np.uint8)
    for u in range(32):
        place = 4 * (u % 8) + u // 8
        for e in range(4):
            code[..., 4 * u + e] = (rows[..., 2 * place + e // 2] >> (4 * (e % 2))) & 15
    return code


def values(rows: np.ndarray, meta: np.ndarray, group: int) -> np.ndarray:
    """float64 values of packed rows and their fp16 (scale, offset) pairs."""
    c = unpack(rows).astype(np.float64)
    m = np.repeat(meta.astype(np.float64), group, axis=-2)
    return m[..., 0] * c + m[..., 1]


def attend(q, K, V, lo, hi, *, pos=None, scale=None, softcap=0.0, bias=None, slopes=None, v_step=None):
    """q [n, Hq, dh], K, V [Hkv, L, dh] (float64), row r sees keys [lo_r, hi_r);
    bias [L] or None, slopes [Hq] or None with positions pos [n].

    Returns (o, spread, noise): the outputs [n, Hq, dh], sum_j w_j a_j per
    element, with a = v_step [Hkv, L, dh] if given and |V| otherwise (what a
    relative error of the weights can move o by), and per (row, head) the
    largest sum_d |q_d k_d| * scale over its visible keys (what the logits'
    own accumulation errors are relative to)."""
    n, hq, dh = q.shape
    hkv, L = K.shape[:2]
    scale = 1.0 / np.sqrt(dh) if scale is None else scale
    a = np.abs(V) if v_step is None else v_step
    o = np.zeros((n, hq, V.shape[-1]))
    spread = np.zeros_like(o)
    noise = np.zeros((n, hq))
    for r in range(n):
        l, h = max(int(lo[r]), 0), min(int(hi[r]), L)
        if l >= h:
            continue
        for i in range(hq):
            k, v = K[i * hkv // hq, l:h], V[i * hkv // hq, l:h]
            x = scale * (k @ q[r, i])
            noise[r, i] = scale * np.max(np.abs(k) @ np.abs(q[r, i]))
            if softcap > 0:
                x = softcap * np.tanh(x / softcap)
            if bias is not None:
                x = x + bias[l:h]
            if slopes is not None:
                x = x - slopes[i] * np.abs(pos[r] - np.arange(l, h))
            w = np.exp(x - x.max())
            w /= w.sum()
            o[r, i] = w @ v
            spread[r, i] = w @ a[i * hkv // hq, l:h]
    return o, spread, noise

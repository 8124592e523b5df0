"""CPU oracle, in binary64, of the operators around a ternary transformer's
projections: rotary positions with several axes, appending to a paged cache and
attention over it -- TEST INFRASTRUCTURE ONLY.

Plain definitions on numpy arrays, one token and one head at a time; nothing is
shared with the product.  Pins in ``tests/test_paged.py``: a quarter turn in
closed form, composition and inverse of rotations, the gradient against central
differences, and attention with one key, equal keys and a two-key logistic.
"""

from __future__ import annotations

import numpy as np


def rotate(x, positions, inv_freq, axis, interleaved=False, inverse=False):
    """x [tokens, heads, dim], positions [tokens, axes] of integers, axis [pairs]."""
    x = np.asarray(x, dtype=np.float64)
    out = x.copy()
    n = len(inv_freq)
    for i in range(n):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        # far positions: the fraction of a turn from exact integer products of the frequency's bits
        angle = np.array([_angle(int(p), float(inv_freq[i])) for p in np.asarray(positions)[:, axis[i]]])[:, None]
        c, s = np.cos(angle), np.sin(angle) * (-1.0 if inverse else 1.0)
        out[:, :, a], out[:, :, b] = x[:, :, a] * c - x[:, :, b] * s, x[:, :, a] * s + x[:, :, b] * c
    return out


def _angle(position, inv_freq):
    """position * inv_freq modulo a turn; the product is formed exactly (extended precision by splitting)."""
    hi = np.float64(np.float32(inv_freq))
    lo = inv_freq - hi
    two_pi = 2 * np.pi
    return float(np.fmod(position * hi, two_pi) + np.fmod(position * lo, two_pi)) if abs(position) < 2 ** 29 else \
        float(position * inv_freq)


def places(q_start, kv_len):
    """(token, sequence, key index) of every new token."""
    for b in range(len(kv_len)):
        n = q_start[b + 1] - q_start[b]
        for i in range(n):
            yield q_start[b] + i, b, kv_len[b] - n + i


def append(cache, x, q_start, kv_len, table):
    """cache [pages, page, heads, dim] with x [tokens, heads, dim] stored (a copy)."""
    out = np.array(cache, dtype=np.float64)
    page = out.shape[1]
    for t, b, j in places(q_start, kv_len):
        if j >= 0:
            out[table[b][j // page], j % page] = x[t]
    return out


def attention(q, k, v, q_start, kv_len, table, scale, window=0, causal=True):
    """Returns (out, weight, spread), all in binary64: out [tokens, heads, dim]; weight, the same with |v| for v (what
    a relative error of the weights is multiplied by); spread [tokens, heads], the largest sum of |q_d k_d| * scale."""
    q = np.asarray(q, dtype=np.float64)
    tokens, heads, dim = q.shape
    page, kv_heads = k.shape[1], k.shape[2]
    group = heads // kv_heads
    out, weight, spread = np.zeros(q.shape), np.zeros(q.shape), np.zeros((tokens, heads))
    held = {}
    for t, b, pos in places(q_start, kv_len):
        hi = pos + 1 if causal else kv_len[b]
        lo = max(0, pos + 1 - window) if window else 0
        if hi <= lo:
            continue
        if b not in held:
            j = np.arange(kv_len[b])
            p = np.asarray(table[b])[j // page]
            held[b] = (np.asarray(k[p, j % page], dtype=np.float64), np.asarray(v[p, j % page], dtype=np.float64))
        ks, vs = held[b][0][lo:hi], held[b][1][lo:hi]
        for h in range(heads):
            g = h // group
            s = ks[:, g] @ q[t, h] * scale
            w = np.exp(s - s.max())
            w /= w.sum()
            out[t, h] = w @ vs[:, g]
            weight[t, h] = w @ np.abs(vs[:, g])
            spread[t, h] = abs(scale) * (np.abs(ks[:, g]) @ np.abs(q[t, h])).max()
    return out, weight, spread

"""Routing, mixtures of ternary experts and sampling in 64 bits (numpy): what the tests compare the library with."""

import numpy as np


def order(values):
    """Indices by value, descending, equal ones by index, NaN last."""
    v = np.where(np.isnan(values), -np.inf, values)
    at = np.arange(len(v))
    return at[np.lexsort((at, np.isnan(values), -v))]


def route(logits, top_k, sigmoid=False, normalize=True, scale=1.0):
    """(experts, weights) [tokens, top_k] of float64 logits."""
    experts = np.stack([order(row)[:top_k] for row in logits]).astype(np.int32)
    with np.errstate(all="ignore"):
        if sigmoid:
            s = 1.0 / (1.0 + np.exp(-logits))
        else:
            z = np.exp(logits - np.max(logits, axis=1, keepdims=True))
            s = z / z.sum(1, keepdims=True)
        s = np.take_along_axis(s, experts.astype(np.int64), 1)
        if normalize:
            s = s / s.sum(1, keepdims=True)
    none = np.all(logits == -np.inf, axis=1)
    if sigmoid:
        none |= np.all(np.take_along_axis(logits, experts.astype(np.int64), 1) == -np.inf, axis=1)
    s[none] = 0.0
    return experts, s * scale


def matrices(soa, experts, rows, cols):
    """float64 [experts, rows, cols] of a ternary weight in the device layout (uint8)."""
    at = experts * rows * cols // 4
    q = soa[:at].reshape(experts, rows, cols // 4)
    c = np.stack([q >> 2 * j & 3 for j in range(4)], -1).reshape(experts, rows, cols).astype(np.float64) - 1.0
    d = soa[at:].view(np.float16).astype(np.float64).reshape(experts, rows, cols // 128)
    return c * np.repeat(d, 128, axis=2)


def silu(z):
    with np.errstate(over="ignore"):
        return z / (1.0 + np.exp(-z))


def experts(gate_up, down, x, expert, weight, residual=None):
    """A mixture's output [tokens, width] for matrices gate_up [experts, 2 ffn, width] and down [experts, width, ffn],
    and what errors in it go by: (out, hidden, sums), where a relative error r of the hidden values moves an element by
    up to r * hidden, and a relative error r of each product summed by up to r * sums."""
    f = down.shape[2]
    out = np.zeros(x.shape) if residual is None else residual.astype(np.float64).copy()
    hidden, sums = np.zeros(x.shape), np.abs(out)
    for e in range(gate_up.shape[0]):
        t, j = np.nonzero(expert == e)
        if not len(t):
            continue
        w = weight[t, j].astype(np.float64)[:, None]
        gu, s = x[t] @ gate_up[e].T, np.abs(x[t]) @ np.abs(gate_up[e]).T
        g, u = gu[:, :f], gu[:, f:]
        h = silu(g) * u
        np.add.at(out, t, w * (h @ down[e].T))
        a = np.abs(down[e]).T
        np.add.at(hidden, t, np.abs(w) * (np.abs(h) @ a))
        # |silu'| < 1.1
        np.add.at(sums, t, np.abs(w) * ((np.abs(h) + 1.1 * np.abs(u) * s[:, :f] + np.abs(silu(g)) * s[:, f:]) @ a))
    return out, hidden, sums


def sample(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, probability, margin) of one row of float64 logits: margin is how far, relative to the kept weight, the
    nearest border (of a cumulative weight to top_p or u, of a weight to min_p) lies from where it would change the
    answer."""
    at = order(logits)
    v = np.where(np.isnan(logits), -np.inf, logits)[at]
    if v[0] == -np.inf:
        return -1, 0.0, 1.0
    margin = 1.0
    if not temperature > 0 or v[0] == np.inf:
        w = (v == v[0]).astype(np.float64)
    else:
        with np.errstate(over="ignore"):
            w = np.exp((v - v[0]) / temperature)
    n = len(w)
    if top_k > 0:
        n = min(n, top_k)
    c = np.cumsum(w[:n])
    if top_p < 1:
        need = max(top_p, 0.0) * c[-1]
        keep = max(1, int(np.sum(c - w[:n] < need)))
        if top_p > 0:
            margin = min(margin, np.min(np.abs(c - need)) / c[-1])
        n = keep
    if min_p > 0:
        least = min(min_p, 1.0)
        margin = min(margin, np.min(np.abs(w[:n] - least)) if least < 1 else 1.0)
        n = max(1, int(np.sum(w[:n] >= least)))
    c = np.cumsum(w[:n])
    u = 0.0 if not u > 0 else min(u, 1 - 2.0 ** -30)
    i = min(int(np.sum(c <= u * c[-1])), int(np.sum(w[:n] > 0)) - 1)
    if u > 0:
        margin = min(margin, np.min(np.abs(c[:-1] - u * c[-1])) / c[-1] if n > 1 else 1.0)
    return int(at[i]), w[i] / c[-1], margin

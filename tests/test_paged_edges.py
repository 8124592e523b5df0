"""Host-side tests (no GPU) of the paged operators' arguments and index arithmetic where they go to their limits."""

import ctypes

import numpy as np
import pytest

from test_paged import fake, index, tq2  # noqa: F401 (fixtures)


@pytest.mark.parametrize("window", [1, 5, 2 ** 62, 2 ** 63 - 2 ** 31, 2 ** 63 - 3, 2 ** 63 - 1])
def test_windows_up_to_64_bits(index, window):  # noqa: F811
    """Tokens before the first key (negative positions) and the widest windows that the call takes."""
    for n, kv, group in ((7, 2, 1), (9, 0, 2), (40, 33, 3), (3, 300, 1)):
        for causal in (0, 1):
            see = [{j for j in range(kv) if (j <= kv - n + i or not causal) and j > kv - n + i - window} for i in range(n)]
            for i in range(n):
                out = (ctypes.c_int * 2)()
                index.keys(n, kv, i, ctypes.c_longlong(window), causal, out)
                assert set(range(out[0], out[1])) == see[i] and out[0] >= 0
            out = (ctypes.c_int * 7)()
            index.item(n, kv, group, 0, 256, ctypes.c_longlong(window), causal, 128, out)
            some = set().union(*see)
            assert out[0] == n * group and out[2] == len({j // 128 for j in some}) and min(out[3:7]) >= 0
            assert set(range(out[3], out[4])) == some or not some


def refused(tq2, q, k, tokens, dim):  # noqa: F811
    """Whether q and k in place, (bytes from a base, heads, token stride, head stride) each, are refused."""
    H, base = tq2.tq2_heads, fake(0)
    rope = tq2.tq2_rope(fake(3), None, dim // 2, 1)
    q, k = (H(base + 4 * at, h, ts, hs, 0) for at, h, ts, hs in (q, k))
    st = tq2.lib.tq2_rope_axes(q, q, k, k, None, None, fake(2), rope, tokens, dim, 0, None)
    assert st != tq2.TQ2_OK and st != tq2.TQ2_ERR_MISALIGNED
    return st == tq2.TQ2_ERR_INVALID_ARG


def cells(view, tokens, dim):
    at, heads, ts, hs = view
    return {at + t * ts + h * hs + d for t in range(tokens) for h in range(heads) for d in range(dim)}


def test_views_that_share_nothing_are_taken_and_others_refused(tq2):  # noqa: F811
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up")
    # q, k, v of each head side by side, [tokens, heads, 3, dim], and heads first, [heads, tokens, 3, dim]
    for ts, hs in ((4 * 3 * 64, 3 * 64), (3 * 64, 10 * 3 * 64)):
        q = (0, 4, ts, hs)
        for at in (64, 128):
            assert not refused(tq2, q, (at, 4, ts, hs), 10, 64)
        assert refused(tq2, q, (63, 4, ts, hs), 10, 64) and refused(tq2, q, (129, 4, ts, hs), 10, 64)
    # grouped: one key head beside every four query heads has no view of one stride; one key head in all has
    assert not refused(tq2, (0, 4, 640, 128), (64, 1, 640, 0), 10, 64)
    rng = np.random.default_rng(9)
    taken = 0
    for _ in range(4000):
        dim, tokens = 2 * int(rng.integers(1, 4)), int(rng.integers(1, 5))
        heads = [int(rng.integers(1, 5)) for _ in range(2)]
        ts, hs = int(rng.integers(0, 40)), int(rng.integers(0, 40))
        views = [(0, heads[0], ts, hs), (int(rng.integers(0, 60)), heads[1], ts, hs)]
        if any(len(cells(v, tokens, dim)) < v[1] * tokens * dim for v in views):
            continue
        if any((tokens > 1 and ts < dim) or (v[1] > 1 and hs < dim) for v in views):
            continue   # (outputs' strides step over what lies below them)
        if any(tokens > 1 and v[1] > 1 and not (ts >= (v[1] - 1) * hs + dim or hs >= (tokens - 1) * ts + dim) for v in views):
            continue
        meet = bool(cells(views[0], tokens, dim) & cells(views[1], tokens, dim))
        assert refused(tq2, *views, tokens, dim) == meet, (views, tokens, dim)
        taken += not meet
    assert taken > 300


# ---------------------------------------------------------------------------
# the weights of the second product


def remainder(w, dtype, terms):
    """What is left of weights w (relative) after so many terms of the type, each the rounding of what the others leave."""
    import torch
    x = torch.as_tensor(w, dtype=torch.float64)
    left = x * (128.0 if dtype == "f16" else 1.0)
    for _ in range(terms):
        left = left - left.to({"f16": torch.float16, "bf16": torch.bfloat16}[dtype]).double()
    return (left.abs() / (x * (128.0 if dtype == "f16" else 1.0))).numpy()


# kept terms and tolerance by type and kernel: half a step to the power of the terms, and 2^-20 for exponent, sums and division
KEPT = {("f16", "few"): (2, 2.0 ** -20), ("bf16", "few"): (3, 2.0 ** -20),
        ("f16", "many"): (2, 2.0 ** -20), ("bf16", "many"): (2, 2.0 ** -16 + 2.0 ** -20)}


def telling_scores(dtype, rows):
    """Scores s = -i/64 whose weight e^s tells whether its last term was kept: without it, it is off by three tolerances."""
    terms, tol = KEPT[dtype, rows]
    s = -np.arange(1, 65) / 64
    return s[remainder(np.exp(s), dtype, terms - 1) > 3 * tol]


@pytest.mark.parametrize("dtype,rows", KEPT, ids=str)
def test_scores_that_tell_whether_a_term_was_kept(dtype, rows):
    """Keys of score 0 and v = 0, every 16th of score s and v = 1: w / (15 + w) is off by more than the tolerance without
    the last term, by less with it."""
    terms, tol = KEPT[dtype, rows]
    s = telling_scores(dtype, rows)
    assert len(s) >= 16
    w = np.exp(s)
    off = 15 / (15 + w)   # d log(w / (15 + w)) / d log w
    assert np.all(remainder(w, dtype, terms - 1) * off > 2 * tol)
    assert np.all(remainder(w, dtype, terms) * off < tol)

"""Host-side tests (no GPU) of the rotary positions, the paged cache and its attention: the oracle's pins, the
fractions of a turn, the index arithmetic that guards the device tables, and every refusal."""

import ctypes
import os
import struct
import subprocess

import numpy as np
import pytest

from oracle import paged

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def tq2():
    import __graft_entry__
    __graft_entry__.build()
    import dit_tq2_g128_gb300 as m
    return m


# ---------------------------------------------------------------------------
# the oracle


def test_rotation_closed_forms():
    x = np.arange(1.0, 9.0).reshape(1, 1, 8)
    quarter = np.array([np.pi / 2, 0.0, np.pi])
    got = paged.rotate(x, [[1]], quarter, [0, 0, 0])[0, 0]
    # pairs (0, 3), (1, 4), (2, 5); 6 and 7 copied
    assert np.allclose(got, [-4, 2, -3, 1, 5, -6, 7, 8], atol=1e-15)
    got = paged.rotate(x, [[1]], quarter, [0, 0, 0], interleaved=True)[0, 0]
    assert np.allclose(got, [-2, 1, 3, 4, -5, -6, 7, 8], atol=1e-15)
    # the axis picks the position
    got = paged.rotate(x, [[0, 1]], quarter, [0, 0, 1])[0, 0]
    assert np.allclose(got, [1, 2, -3, 4, 5, -6, 7, 8], atol=1e-15)


def test_rotations_compose_and_invert():
    rng = np.random.default_rng(0)
    x, f = rng.standard_normal((5, 2, 10)), rng.random(5)
    p = rng.integers(-50, 50, (5, 2))
    axis = [0, 1, 1, 0, 1]
    once = paged.rotate(x, p, f, axis)
    assert np.allclose(paged.rotate(once, p, f, axis, inverse=True), x, atol=1e-13)
    assert np.allclose(paged.rotate(once, 2 * p, f, axis), paged.rotate(x, 3 * p, f, axis), atol=1e-13)


@pytest.mark.parametrize("interleaved", [False, True])
def test_inverse_is_the_gradient(interleaved):
    rng = np.random.default_rng(1)
    x, g = rng.standard_normal((2, 3, 1, 9))
    p, f, axis = rng.integers(0, 1000, (3, 2)), rng.random(4), [0, 1, 0, 1]
    grad = paged.rotate(g, p, f, axis, interleaved, inverse=True)
    for i in np.ndindex(x.shape):
        e = np.zeros(x.shape)
        e[i] = 0.5  # linear: differences are exact up to rounding
        up, down = (paged.rotate(x + s * e, p, f, axis, interleaved) for s in (1, -1))
        assert abs(np.sum(g * (up - down)) - grad[i]) < 1e-12


def test_attention_closed_forms():
    rng = np.random.default_rng(2)
    k, v = rng.standard_normal((2, 3, 4, 1, 8))
    q = rng.standard_normal((2, 2, 8))
    out, _, _ = paged.attention(q[:1], k, v, [0, 1], [1], [[2]], 0.3)
    assert np.allclose(out[0], v[2, 0])                                   # one key
    out, _, _ = paged.attention(q[:1], 0 * k, v, [0, 1], [6], [[2, 0]], 0.3)
    assert np.allclose(out[0], np.concatenate([v[2], v[0, :2]])[:, 0].mean(0))  # equal keys
    out, _, _ = paged.attention(q, k, v, [0, 2], [2], [[1]], 0.3)
    w = 1 / (1 + np.exp(-0.3 * (q[1] @ (k[1, 1, 0] - k[1, 0, 0]))))
    assert np.allclose(out[1], (1 - w)[:, None] * v[1, 0, 0] + w[:, None] * v[1, 1, 0])
    assert np.allclose(out[0], v[1, 0])                                   # the first token sees one key
    out, _, _ = paged.attention(q, k, v, [0, 2], [1], [[1]], 0.3)
    assert np.all(out[0] == 0) and np.allclose(out[1], v[1, 0])           # a token before every key


# ---------------------------------------------------------------------------
# fractions of a turn


def test_rope_turns_are_the_fractions(tq2):
    from fractions import Fraction
    f = np.array([0.0, 1.0, 1e-7, 2 * np.pi, 3.5 * np.pi, -0.25, 1e4, np.pi, 5e-324])
    turns = tq2.tq2_rope_turns(f)
    for x, t in zip(f, turns):
        want = Fraction(float(x / (2 * np.pi))) % 1
        got = Fraction(int(t), 2 ** 64)
        d = abs(got - want)
        assert min(d, 1 - d) <= Fraction(1, 2 ** 65), x


def test_far_positions_keep_their_angle(tq2):
    f = 10_000.0 ** (-np.arange(64) / 64)
    turns = tq2.tq2_rope_turns(f)
    for pos in (1, 12_345, (1 << 20) + 3, -77_777):
        phase = np.array([(pos * int(t)) % 2 ** 64 for t in turns], dtype=np.float64) / 2 ** 64
        want = pos * f
        assert np.max(np.abs(np.exp(2j * np.pi * phase) - np.exp(1j * want))) < 1e-9


# ---------------------------------------------------------------------------
# the index arithmetic behind the device tables


@pytest.fixture(scope="module")
def index(tmp_path_factory):
    d = tmp_path_factory.mktemp("paged_index")
    src = d / "probe.cpp"
    src.write_text("""
#include "paged_index.h"
using namespace tq2;
extern "C" {
static BatchView view(const int *qs, const int *kl, const int *pt, const long long *n) {
    return BatchView{qs, kl, pt, n[0], n[1], n[2], int(n[3]), int(n[4]), int(n[5]), int(n[6])};
}
int span(const int *qs, const int *kl, const int *pt, const long long *n, int b, int *out) {
    bool bad = false;
    const SeqSpan s = seq_span(view(qs, kl, pt, n), b, bad);
    out[0] = s.q0, out[1] = s.n, out[2] = s.kv;
    return bad;
}
long long page(const int *qs, const int *kl, const int *pt, const long long *n, int b, int entry, int *bad) {
    bool w = false;
    const long long p = page_of(view(qs, kl, pt, n), b, entry, w);
    *bad = w;
    return p;
}
int seq(const int *qs, const int *kl, const int *pt, const long long *n, long long t) {
    return seq_of(view(qs, kl, pt, n), t);
}
void keys(int n, int kv, int i, long long window, int causal, int *out) {
    const KeyRange r = keys_of(SeqSpan{0, n, kv}, i, window, causal);
    out[0] = r.lo, out[1] = r.hi;
}
void boxes(int from, int keys, int rows, int first, int last, int *out) {
    const BoxRange r = boxes_of(from, keys, rows, first, last);
    out[0] = r.lo, out[1] = r.hi;
}
void tiles(int n, int kv, long long window, int causal, int keys, int split, int *out) {
    const TileSpan t = tiles_of(SeqSpan{0, n, kv}, window, causal, keys, split);
    out[0] = t.tile0, out[1] = t.tiles, out[2] = t.units;
}
int item(int n, int kv, int group, int row0, int most, long long window, int causal, int keys, int *out) {
    const ItemSpan t = item_span(SeqSpan{0, n, kv}, group, row0, most, window, causal, keys);
    out[0] = t.rows, out[1] = t.block0, out[2] = t.blocks;
    out[3] = t.see.lo, out[4] = t.see.hi, out[5] = t.see.lo_all, out[6] = t.see.hi_all;
    return 0;
}
}
""")
    lib = d / "probe.so"
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I",
                    os.path.join(ROOT, "dit_tq2_g128_gb300", "csrc"), str(src), "-o", str(lib)], check=True)
    L = ctypes.CDLL(str(lib))
    L.page.restype = ctypes.c_longlong
    return L


class Tables:
    def __init__(self, q_start, kv_len, table, tokens, pages, max_q, max_kv, page_size):
        self.a = [np.ascontiguousarray(x, dtype=np.int32) for x in (q_start, kv_len, table)]
        self.n = np.array([tokens, self.a[2].shape[1], pages, len(kv_len), max_q, max_kv, page_size], dtype=np.int64)
        self.p = [x.ctypes.data_as(ctypes.c_void_p) for x in (*self.a, self.n)]


def test_spans_are_clamped(index):
    rng = np.random.default_rng(3)
    wild = [0, 1, 5, 7, 20, -1, -2 ** 31, 2 ** 31 - 1, 100]
    for _ in range(3000):
        seqs, tokens, max_q, max_kv, entries, page = rng.integers(1, 9, 6)
        t = Tables(rng.choice(wild, seqs + 1), rng.choice(wild, seqs), rng.choice(wild, (seqs, entries)), tokens, 4,
                   max_q, max_kv, page)
        for b in range(seqs):
            out = (ctypes.c_int * 3)()
            bad = index.span(*t.p, b, out)
            q0, n, kv = out
            assert 0 <= q0 and 0 <= n <= max_q and q0 + n <= tokens and 0 <= kv <= min(max_kv, entries * page)
            fine = (0 <= t.a[0][b] <= t.a[0][b + 1] <= tokens and t.a[0][b + 1] - t.a[0][b] <= max_q
                    and 0 <= t.a[1][b] <= min(max_kv, entries * page))
            assert bool(bad) == (not fine)
            if fine:
                assert (q0, n, kv) == (t.a[0][b], t.a[0][b + 1] - t.a[0][b], t.a[1][b])
            for e in range(entries):
                w = ctypes.c_int()
                p = index.page(*t.p, b, e, ctypes.byref(w))
                assert p == (t.a[2][b, e] if 0 <= t.a[2][b, e] < 4 else -1) and bool(w.value) == (p < 0)
        for tok in range(tokens):
            assert -1 <= index.seq(*t.p, ctypes.c_longlong(tok)) < seqs


def test_every_token_finds_its_sequence(index):
    rng = np.random.default_rng(4)
    for _ in range(500):
        n = rng.integers(0, 5, rng.integers(1, 40))
        q_start = np.concatenate([[0], np.cumsum(n)])
        pad = int(rng.integers(0, 3))
        t = Tables(q_start, np.ones(len(n)), np.zeros((len(n), 1)), int(q_start[-1]) + pad, 1, max(1, n.max()), 9, 1)
        want = np.repeat(np.arange(len(n)), n)
        for tok in range(int(q_start[-1]) + pad):
            assert index.seq(*t.p, ctypes.c_longlong(tok)) == (want[tok] if tok < len(want) else -1)


def test_visible_keys(index):
    for n, kv in ((1, 0), (1, 1), (4, 9), (6, 3), (3, 3)):
        for i in range(n):
            for window in (0, 1, 2, 5, 1 << 60):
                for causal in (0, 1):
                    out = (ctypes.c_int * 2)()
                    index.keys(n, kv, i, ctypes.c_longlong(window), causal, out)
                    pos = kv - n + i
                    want = [j for j in range(kv) if (j <= pos or not causal) and (j > pos - window or not window)]
                    assert list(range(out[0], out[1])) == want


def test_boxes_of_a_tile(index):
    """The boxes that are counted are those that hold a key, in tiles that hold none too."""
    rng = np.random.default_rng(5)
    for _ in range(4000):
        keys = int(rng.choice([64, 128]))
        rows = 1 << int(rng.integers(0, 7 if keys == 64 else 8))
        first = int(rng.integers(0, 700))
        last = first + int(rng.integers(0, 500))
        start = int(rng.integers(0, 10)) * keys
        out = (ctypes.c_int * 2)()
        index.boxes(start, keys, rows, first, last, out)
        want = [i for i in range(keys // rows)
                if any(first <= k < last for k in range(start + i * rows, start + (i + 1) * rows))]
        assert list(range(out[0], out[1])) == want


def test_tiles_of_a_span(index):
    rng = np.random.default_rng(7)
    for _ in range(2000):
        n, kv, window = int(rng.integers(0, 40)), int(rng.integers(0, 600)), int(rng.choice([0, 1, 5, 64, 65, 300, 10 ** 9]))
        for causal in (0, 1):
            seen = sorted({j for i in range(n) for j in range(kv)
                           if (j <= kv - n + i or not causal) and (j > kv - n + i - window or not window)})
            for split in (0, 1):
                out = (ctypes.c_int * 3)()
                index.tiles(n, kv, ctypes.c_longlong(window), causal, 64, split, out)
                want = sorted({j // 64 for j in seen})
                assert out[1] == len(want) and (not want or out[0] == want[0])
                assert out[2] == (0 if n == 0 else max(1, len(want)) if split else 1)


def test_items_of_a_span(index):
    rng = np.random.default_rng(6)
    for _ in range(1500):
        n, kv, group = int(rng.integers(1, 60)), int(rng.integers(0, 600)), int(rng.integers(1, 17))
        window = int(rng.choice([0, 1, 7, 128, 300]))
        most = 64
        for causal in (0, 1):
            for row0 in range(0, n * group, most):
                out = (ctypes.c_int * 7)()
                index.item(n, kv, group, row0, most, ctypes.c_longlong(window), causal, 128, out)
                rows = range(row0, min(n * group, row0 + most))
                assert out[0] == len(rows)
                see = [{j for j in range(kv) if (j <= kv - n + i or not causal) and (j > kv - n + i - window or not window)}
                       for i in sorted({r // group for r in rows})]
                some, every = set().union(*see), set.intersection(*see)
                assert set(range(out[3], out[4])) == some or (not some and out[2] == 0)
                if all(see):
                    assert set(range(out[5], out[6])) == every
                want = sorted({j // 128 for j in some})
                assert out[2] == len(want) and (not want or out[1] == want[0])


# ---------------------------------------------------------------------------
# refusals


A = 1 << 30  # fake device addresses, 1 GiB apart


def fake(i):
    return (i + 1) * A


def test_rope_refusals(tq2):
    bad, skew = tq2.TQ2_ERR_INVALID_ARG, tq2.TQ2_ERR_MISALIGNED
    H = tq2.tq2_heads

    def call(q=H(fake(0), 4, 512, 128, 0), qo=H(fake(1), 4, 512, 128, 0), k=None, ko=None, v=None, vo=None,
             pos=fake(2), rope=tq2.tq2_rope(fake(3), fake(4), 64, 3), tokens=10, dim=128):
        return tq2.lib.tq2_rope_axes(q, qo, k, ko, v, vo, pos, rope, tokens, dim, 0, None)

    assert call(tokens=0) == tq2.TQ2_OK and call(tokens=0, q=None, qo=None) == tq2.TQ2_OK
    assert call(tokens=-1) == bad and call(tokens=1 << 31) == bad and call(dim=0) == bad and call(dim=65537) == bad
    assert call(rope=None) == bad and call(q=None) == bad and call(qo=None) == bad
    assert call(rope=tq2.tq2_rope(fake(3), None, 65, 1)) == bad           # 2 pairs > dim
    assert call(rope=tq2.tq2_rope(fake(3), None, -1, 1)) == bad
    for axes in (0, 17, -1):
        assert call(rope=tq2.tq2_rope(fake(3), None, 64, axes)) == bad
    assert call(rope=tq2.tq2_rope(None, None, 64, 1)) == bad and call(pos=None) == bad
    assert call(rope=tq2.tq2_rope(fake(3) + 4, None, 64, 1)) == skew and call(pos=fake(2) + 4) == skew
    assert call(k=H(fake(5), 1, 128, 128, 0)) == bad and call(ko=H(fake(5), 1, 128, 128, 0)) == bad
    assert call(v=H(fake(5), 1, 128, 128, 0)) == bad
    assert call(qo=H(fake(1), 5, 640, 128, 0)) == bad                      # heads differ
    assert call(k=H(fake(5), 1, 128, 128, 1), ko=H(fake(6), 1, 128, 128, 0)) == bad   # types differ
    assert call(k=H(fake(5), 1, 128, 128, 0), ko=H(fake(6), 1, 128, 128, 1)) == bad
    assert call(q=H(fake(0), 4, 512, 128, 3)) == bad and call(q=H(fake(0), 0, 512, 128, 0)) == bad
    assert call(q=H(fake(0), 4, -512, 128, 0)) == bad and call(q=H(0, 4, 512, 128, 0)) == bad
    assert call(q=H(fake(0), 20000, 512, 128, 0)) == bad
    assert call(q=H(fake(0) + 2, 4, 512, 128, 0)) == skew
    # outputs whose elements coincide
    assert call(qo=H(fake(1), 4, 512, 127, 0)) == bad and call(qo=H(fake(1), 4, 511, 128, 0)) == bad
    assert call(qo=H(fake(1), 4, 0, 128, 0)) == bad
    # overlaps
    assert call(qo=H(fake(0) + 16, 4, 512, 128, 0)) == bad
    assert call(qo=H(fake(2) // 2, 4, 512, 128, 0), k=H(fake(2) // 2 + 512, 4, 512, 128, 0),
                ko=H(fake(6), 4, 512, 128, 0)) == bad


def test_slices_of_one_projection_are_apart(tq2):
    # q in place in the columns [0, 512) of rows of 768, k in [512, 640): no refusal before the device is looked at
    H, base = tq2.tq2_heads, fake(0)
    rope = tq2.tq2_rope(fake(3), None, 64, 1)
    q, k = H(base, 4, 768, 128, 0), H(base + 4 * 512, 1, 768, 128, 0)
    st = tq2.lib.tq2_rope_axes(q, q, k, k, None, None, fake(2), rope, 10, 128, 0, None)
    import torch
    if not torch.cuda.is_available():
        assert st not in (tq2.TQ2_OK, tq2.TQ2_ERR_INVALID_ARG, tq2.TQ2_ERR_MISALIGNED)
    k = H(base + 4 * 511, 1, 768, 128, 0)  # one element into q's columns
    assert tq2.lib.tq2_rope_axes(q, q, k, k, None, None, fake(2), rope, 10, 128, 0, None) == tq2.TQ2_ERR_INVALID_ARG
    k = H(base + 4 * 641, 1, 768, 128, 0)  # wraps into the next row's q
    assert tq2.lib.tq2_rope_axes(q, q, k, k, None, None, fake(2), rope, 10, 128, 0, None) == tq2.TQ2_ERR_INVALID_ARG


def cache(tq2, k=None, v=None, pages=8, page=16, heads=2, dim=128, s=None, dtype=1):
    s = s or (page * heads * dim, heads * dim, dim)
    return tq2.tq2_kv_cache(fake(10) if k is None else k, fake(11) if v is None else v, pages, page, heads, dim, *s,
                            dtype)


def batch(tq2, qs=None, kl=None, pt=None, seqs=2, tokens=10, max_q=6, max_kv=50, stride=4):
    return tq2.tq2_batch(fake(12) if qs is None else qs, fake(13) if kl is None else kl,
                         fake(14) if pt is None else pt, seqs, tokens, max_q, max_kv, stride)


def bad_caches(tq2):
    bad, skew = tq2.TQ2_ERR_INVALID_ARG, tq2.TQ2_ERR_MISALIGNED
    yield None, bad
    for kw in (dict(k=0), dict(v=0), dict(dtype=0), dict(dtype=3), dict(dim=0), dict(dim=132), dict(dim=136),
               dict(dim=20), dict(heads=0), dict(pages=0), dict(pages=1 << 31), dict(page=0), dict(page=(1 << 20) + 1),
               dict(s=(4096, 256, 120)), dict(s=(4096, 248, 128)), dict(s=(4000, 256, 128)), dict(s=(-8, 256, 128)),
               dict(s=(0, 256, 128))):
        yield cache(tq2, **kw), bad
    for kw in (dict(k=fake(10) + 8), dict(v=fake(11) + 2), dict(s=(8192, 260, 128)), dict(s=(4100, 256, 128)),
               dict(s=(8448, 264, 132))):
        yield cache(tq2, **kw), skew


def bad_batches(tq2):
    bad, skew = tq2.TQ2_ERR_INVALID_ARG, tq2.TQ2_ERR_MISALIGNED
    yield None, bad
    for kw in (dict(qs=0), dict(kl=0), dict(pt=0), dict(seqs=-1), dict(seqs=(1 << 20) + 1), dict(tokens=-1),
               dict(tokens=(1 << 30) + 1), dict(max_q=-1), dict(max_kv=-1), dict(max_kv=1 << 31), dict(stride=-1)):
        yield batch(tq2, **kw), bad
    for kw in (dict(qs=fake(12) + 2), dict(kl=fake(13) + 1), dict(pt=fake(14) + 2)):
        yield batch(tq2, **kw), skew


def test_append_refusals(tq2):
    bad, skew, H = tq2.TQ2_ERR_INVALID_ARG, tq2.TQ2_ERR_MISALIGNED, tq2.tq2_heads
    k, v = H(fake(0), 2, 256, 128, 0), H(fake(1), 2, 256, 128, 0)
    q, qo = H(fake(2), 8, 1024, 128, 0), H(fake(3), 8, 1024, 128, 1)
    good_c, good_b = cache(tq2), batch(tq2)

    def call(q=q, qo=qo, k=k, v=v, pos=None, rope=tq2.tq2_rope(fake(4), None, 64, 1), b=good_b, c=good_c):
        return tq2.lib.tq2_kv_append(q, qo, k, v, pos, rope, b, c, None)

    for c, why in bad_caches(tq2):
        assert call(c=c) == why
    for b, why in bad_batches(tq2):
        assert call(b=b) == why
    for b in (batch(tq2, seqs=0), batch(tq2, tokens=0), batch(tq2, max_q=0), batch(tq2, tokens=0, qs=0, kl=0, pt=0)):
        assert call(b=b) == tq2.TQ2_OK and call(b=b, k=None, v=None) == tq2.TQ2_OK
    assert call(k=None) == bad and call(v=None) == bad and call(q=None) == bad and call(qo=None) == bad
    assert call(k=H(fake(0), 3, 384, 128, 0)) == bad and call(v=H(fake(1), 2, 256, 128, 1)) == bad
    assert call(q=H(fake(2), 8, 1024, 128, 2)) == bad and call(qo=H(fake(3), 8, 1024, 128, 0)) == bad
    assert call(qo=H(fake(3), 7, 1024, 128, 1)) == bad and call(qo=H(fake(3), 8, 0, 128, 1)) == bad
    assert call(rope=tq2.tq2_rope(fake(4), None, 64, 3)) == bad   # three axes need positions
    assert call(rope=tq2.tq2_rope(fake(4), None, 65, 1)) == bad
    assert call(rope=tq2.tq2_rope(0, None, 64, 1)) == bad
    assert call(k=H(fake(10), 2, 256, 128, 0)) == bad             # input in the cache
    assert call(qo=H(fake(11), 8, 1024, 128, 1)) == bad
    assert call(qo=H(fake(0), 8, 1024, 128, 1)) == bad            # q_out over k
    assert call(k=H(fake(0) + 2, 2, 256, 128, 0)) == skew


def test_attention_refusals(tq2):
    bad, skew, H = tq2.TQ2_ERR_INVALID_ARG, tq2.TQ2_ERR_MISALIGNED, tq2.tq2_heads
    q, out = H(fake(0), 8, 1024, 128, 1), H(fake(1), 8, 1024, 128, 1)
    good_c, good_b = cache(tq2), batch(tq2)

    def call(q=q, out=out, c=good_c, b=good_b, scale=0.1, window=0, ws=None, nws=0):
        return tq2.lib.tq2_attention_paged(q, out, c, b, scale, window, 1, ws, nws, None)

    for c, why in bad_caches(tq2):
        assert call(c=c) == why
    for b, why in bad_batches(tq2):
        assert call(b=b) == why
    for b in (batch(tq2, seqs=0), batch(tq2, tokens=0), batch(tq2, max_q=0)):
        assert call(b=b) == tq2.TQ2_OK and call(b=b, q=None, out=None) == tq2.TQ2_OK
    assert call(q=None) == bad and call(out=None) == bad
    assert call(scale=float("nan")) == bad and call(scale=float("inf")) == bad and call(window=-1) == bad
    assert call(q=H(fake(0), 7, 1024, 128, 1), out=H(fake(1), 7, 1024, 128, 1)) == bad   # 7 over 2 key heads
    assert call(out=H(fake(1), 6, 1024, 128, 1)) == bad
    assert call(q=H(fake(0), 8, 1024, 128, 2)) == bad and call(q=H(fake(0), 8, 1024, 128, 0)) == bad
    assert call(out=H(fake(1), 8, 1024, 128, 2)) == bad
    assert call(out=H(fake(1), 8, 0, 128, 1)) == bad and call(out=H(fake(0), 8, 1024, 128, 1)) == bad
    assert call(out=H(fake(10), 8, 1024, 128, 1)) == bad and call(out=H(fake(11), 8, 1024, 128, 1)) == bad
    assert call(q=H(fake(0) + 8, 8, 1024, 128, 1)) == skew and call(q=H(fake(0), 8, 1028, 128, 1)) == skew
    assert call(out=H(fake(1), 8, 1040, 130, 1)) == skew
    big = batch(tq2, seqs=1, tokens=1, max_q=1, max_kv=1 << 20, stride=1 << 16)
    need = tq2.tq2_attention_paged_workspace_bytes(8, good_c, big)
    one = H(fake(0), 8, 1024, 128, 1)
    if need:
        assert call(q=one, b=big, ws=fake(20), nws=need - 1) == bad
        assert call(q=one, b=big, ws=fake(20) + 8, nws=need) == skew
        assert call(q=one, b=big, ws=fake(0), nws=need) == bad
        assert call(q=one, b=big, ws=fake(10), nws=need) == bad


def test_workspace_of_invalid_arguments_is_zero(tq2):
    f = tq2.tq2_attention_paged_workspace_bytes
    c, b = cache(tq2), batch(tq2)
    assert f(7, c, b) == 0 and f(0, c, b) == 0 and f(8, None, b) == 0 and f(8, c, None) == 0
    assert f(8, c, batch(tq2, tokens=0)) == 0 and f(8, c, batch(tq2, seqs=-1)) == 0


def test_strides_of_single_elements_say_nothing(tq2):
    # one page of one slot with one head: any strides are those of a cache
    import torch
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up")
    c = cache(tq2, pages=1, page=1, heads=1, s=(3, 5, 7))
    H = tq2.tq2_heads
    one = H(fake(0), 1, 9, 11, 1)
    b = batch(tq2, seqs=1, tokens=1, max_q=1, max_kv=1, stride=1)
    st = tq2.lib.tq2_attention_paged(one, H(fake(1), 1, 9, 11, 1), c, b, 0.1, 0, 1, None, 0, None)
    assert st not in (tq2.TQ2_OK, tq2.TQ2_ERR_INVALID_ARG, tq2.TQ2_ERR_MISALIGNED)


def test_packed_structs_have_the_headers_layout(tq2, tmp_path):
    src = tmp_path / "s.c"
    src.write_text('#include "tq2.h"\n#include <stdio.h>\nint main(void) { printf("%zu %zu %zu %zu %zu %zu %zu", '
                   "sizeof(tq2_heads), sizeof(tq2_rope), sizeof(tq2_kv_cache), sizeof(tq2_batch), "
                   "offsetof(tq2_heads, dtype), offsetof(tq2_rope, interleaved), offsetof(tq2_kv_cache, dtype)); }")
    exe = tmp_path / "s"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], capture_output=True, check=True, text=True).stdout.split()]
    assert got == [len(tq2.tq2_heads(0, 1, 1, 1, 0)), len(tq2.tq2_rope(0, 0, 0)), len(cache(tq2)), len(batch(tq2)),
                   32, 28, 72]
    assert struct.calcsize("=qqqqi4x") == 40


def test_tensor_level_refusals(tq2):
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("checked without a device")
    k = torch.zeros(4, 16, 2, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        tq2.KVCache(k, k)                                      # host memory
    with pytest.raises(ValueError):
        tq2.KVCache(k, k[:2])
    with pytest.raises(ValueError):
        tq2.PagedBatch(torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
                       torch.zeros(2, 4, dtype=torch.int32), tokens=2, max_q=1, max_kv=64)
    with pytest.raises(ValueError):
        tq2.Rope([1.0, 0.5], axis=[0, 2], axes=2, device="cpu")
    with pytest.raises(tq2.TQ2Error):
        tq2.Rope([1.0, float("inf")], device="cpu")
    r = tq2.Rope([1.0, 0.5], axis=[0, 1], axes=2, device="cpu")
    assert r.pairs == 2 and len(r.packed) == 32

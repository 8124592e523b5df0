"""GPU tests of the rotary positions, the paged append and the paged attention against the binary64 oracle.

Tolerances count roundings.  A rotation: one rounding to the output's type (eps/2) and an absolute 2^-21 of |a| + |b|
for the f32 sines, products and sum.  Attention: one rounding of the output; the weights' rounding in the second
product (eps/2 of the cache's type; its square for an f32 output, whose weights are two terms; 2^-25 a key for
binary16's subnormals); f32 scores (dim + 8 roundings of at most their spread, on both sides of the exponential),
exponential and sums (2^-20 and 2^-23 a key)."""

import numpy as np
import pytest

from oracle import paged

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def tq2():
    import dit_tq2_g128_gb300 as m
    return m


@pytest.fixture(autouse=True)
def status_is_clean(tq2):
    yield
    assert tq2.tq2_device_status() == tq2.TQ2_OK


def half_step(dtype):
    return torch.finfo(DT[dtype]).eps / 2


def tiny(dtype):
    return 2.0 ** -25 if dtype == "f16" else 1e-30


def host(t):
    return t.detach().double().cpu().numpy()


def check(got, want, tol, what=""):
    got = host(got)
    assert got.shape == want.shape
    fine = np.isfinite(want)
    assert np.array_equal(np.isfinite(got), fine), f"{what}: other values are finite"
    err = np.abs(np.where(fine, got - np.where(fine, want, 0), 0))
    over = err / np.where(fine, tol, 1)
    at = np.unravel_index(np.argmax(over), over.shape) if over.size else ()
    assert not over.size or over[at] <= 1, f"{what}: error {err[at]:.3g} of {tol[at]:.3g} at {at}"


# ---------------------------------------------------------------------------
# rotary positions


def rope_tol(x, pairs, interleaved, want, dtype):
    x = np.abs(x)
    near = x.copy()
    n = pairs
    a = (slice(None), slice(None), slice(0, 2 * n, 2)) if interleaved else (slice(None), slice(None), slice(0, n))
    b = (slice(None), slice(None), slice(1, 2 * n, 2)) if interleaved else (slice(None), slice(None), slice(n, 2 * n))
    near[a] = near[b] = x[a] + x[b]
    near[:, :, 2 * n:] = 0
    return half_step(dtype) * np.abs(want) * (1 + 2.0 ** -9) + 2.0 ** -21 * near + tiny(dtype)


def frequencies(pairs, axes, rng, mixed):
    f = 10_000.0 ** (-np.arange(pairs) / max(1, pairs))
    axis = rng.integers(0, axes, pairs) if mixed else np.arange(pairs) * axes // max(1, pairs)
    return f, axis


def layout(shape, kind, dtype, gen=None, extra=0):
    """A [tokens, heads, dim] view: contiguous rows, heads first, or a slice of wider rows (offset by `extra`)."""
    t, h, d = shape
    make = (lambda s: torch.randn(s, device="cuda", generator=gen).to(DT[dtype])) if gen is not None else \
        (lambda s: torch.full(s, float("nan"), device="cuda", dtype=DT[dtype]))
    if kind == "rows":
        return make((t, h, d))
    if kind == "heads":
        return make((h, t, d)).transpose(0, 1)
    return make((t, (h + 2) * d + extra))[:, d + extra:d + extra + h * d].unflatten(1, (h, d))


ROPE = [
    # tokens, heads, kv heads, dim, pairs, axes, interleaved, mixed axes
    (1, 1, 1, 2, 1, 1, False, False),
    (1, 3, 1, 128, 64, 3, True, False),
    (7, 5, 2, 128, 64, 4, False, True),
    (33, 9, 3, 128, 32, 1, True, False),
    (65, 4, 4, 80, 40, 2, False, False),
    (19, 2, 1, 72, 36, 3, False, True),
    (20, 3, 2, 72, 12, 1, True, False),
    (5, 17, 1, 96, 31, 2, False, True),
    (6, 2, 2, 67, 20, 3, True, True),
    (4, 1, 1, 64, 0, 1, False, False),
    (300, 24, 24, 128, 64, 4, True, False),
    (3, 2, 1, 1000, 500, 2, True, False),
]


@pytest.mark.parametrize("case", ROPE, ids=str)
@pytest.mark.parametrize("io", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f16"), ("f32", "bf16"), ("f16", "f32"),
                                ("bf16", "f16")], ids=str)
@pytest.mark.parametrize("way", [("rows", "heads", 0, False), ("heads", "slice", 0, True), ("slice", "rows", 3, False)],
                         ids=str)
def test_rope(tq2, case, io, way):
    tokens, heads, kv_heads, dim, pairs, axes, interleaved, mixed = case
    src, dst, extra, inverse = way
    rng = np.random.default_rng(tokens + dim)
    gen = torch.Generator(device="cuda").manual_seed(dim + tokens)
    f, axis = frequencies(pairs, axes, rng, mixed)
    pos = rng.integers(-100, 5000, (tokens, axes))
    xs = [layout((tokens, h, dim), src, io[0], gen, extra) for h in (heads, kv_heads, kv_heads)]
    outs = [layout((tokens, h, dim), dst, io[1], None, extra) for h in (heads, kv_heads, kv_heads)]
    rope = tq2.Rope(f, axis if axes > 1 else None, axes=axes, interleaved=interleaved)
    got = tq2.rope_axes(*xs, positions=torch.from_numpy(pos).cuda(), rope=rope, out=outs, inverse=inverse)
    for x, o, turned in zip(xs, got, (True, True, False)):
        want = paged.rotate(host(x), pos, f if turned else [], axis, interleaved, inverse)
        check(o, want, rope_tol(host(x), pairs if turned else 0, interleaved, want, io[1]), str(turned))


def test_rope_far_positions_and_in_place(tq2):
    rng = np.random.default_rng(5)
    gen = torch.Generator(device="cuda").manual_seed(5)
    f, _ = frequencies(64, 1, rng, False)
    pos = np.array([[0], [1], [99_999], [(1 << 20) + 7], [-(1 << 20)], [10_000_019]])
    fused = torch.randn((6, 5 * 128), device="cuda", generator=gen)
    before = host(fused).reshape(6, 5, 128)
    q, k = fused[:, :384].unflatten(1, (3, 128)), fused[:, 384:].unflatten(1, (2, 128))
    rope = tq2.Rope(f)
    tq2.rope_axes(q, k, positions=torch.from_numpy(pos).cuda(), rope=rope, out=(q, k))
    want = paged.rotate(before, pos, f, [0] * 64)
    check(fused.view(6, 5, 128), want, rope_tol(before, 64, False, want, "f32"))
    # the gradient undoes it
    tq2.rope_axes(q, k, positions=torch.from_numpy(pos).cuda(), rope=rope, out=(q, k), inverse=True)
    check(fused.view(6, 5, 128), before, 2 * rope_tol(before, 64, False, before, "f32"))


def test_rope_broadcast_input(tq2):
    # one head's values read by every head (stride 0), as a shared key's gradient sources are
    gen = torch.Generator(device="cuda").manual_seed(6)
    x = torch.randn((9, 1, 64), device="cuda", generator=gen).expand(9, 4, 64)
    f, _ = frequencies(32, 1, None, False)
    pos = np.arange(9).reshape(9, 1)
    out, = tq2.rope_axes(x, positions=torch.from_numpy(pos).cuda(), rope=tq2.Rope(f))
    want = paged.rotate(host(x), pos, f, [0] * 32)
    check(out, want, rope_tol(host(x), 32, False, want, "f32"))


def test_rope_gradient_against_differences(tq2):
    gen = torch.Generator(device="cuda").manual_seed(7)
    x, g, d = torch.randn((3, 11, 2, 48), device="cuda", generator=gen)
    f, axis = frequencies(20, 2, None, False)
    pos = torch.arange(22, device="cuda").view(11, 2)
    rope = tq2.Rope(f, axis, axes=2)
    up, = tq2.rope_axes(x + d, positions=pos, rope=rope)
    down, = tq2.rope_axes(x - d, positions=pos, rope=rope)
    grad, = tq2.rope_axes(g, positions=pos, rope=rope, inverse=True)
    lhs, rhs = (g.double() * (up.double() - down.double())).sum() / 2, (grad.double() * d.double()).sum()
    # f32 roundings of x +- d and of each rotation, at most 2^-20 of the values' magnitudes
    assert abs(lhs - rhs) <= 2.0 ** -20 * (g.abs() * (x.abs() + d.abs()) * 4).sum() + 2.0 ** -20 * (g.abs() * d.abs() * 4).sum()


# ---------------------------------------------------------------------------
# a step over a paged cache


class Step:
    """Tables, cache and oracle inputs of one step; slots that hold no key are filled with `rest`."""

    def __init__(self, tq2, q_len, kv_len, kv_heads, dim, page, order="slots", dtype="f16", seed=0, rest=float("nan"),
                 pad=0):
        rng = np.random.default_rng(seed)
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.q_len, self.kv_len, self.dtype, self.dim, self.page = q_len, kv_len, dtype, dim, page
        need = [-(-n // page) for n in kv_len]
        pages = sum(need) + 2
        ids = rng.permutation(pages)
        entries = max(1, max(need))
        self.table = np.full((len(kv_len), entries), -7, dtype=np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n
        self.q_start = np.concatenate([[0], np.cumsum(q_len)]).astype(np.int32)
        self.tokens = int(self.q_start[-1]) + pad
        shape = (pages, page, kv_heads, dim) if order == "slots" else (pages, kv_heads, page, dim)

        def plane():
            p = torch.full(shape, rest, device="cuda", dtype=DT[dtype])
            return p if order == "slots" else p.transpose(1, 2)

        self.k, self.v = plane(), plane()
        for b, n in enumerate(kv_len):
            if n:
                j = torch.arange(n, device="cuda")
                p, o = torch.from_numpy(self.table[b].astype(np.int64)).cuda()[j // page], j % page
                for c in (self.k, self.v):
                    c[p, o] = torch.randn((n, kv_heads, dim), device="cuda", generator=self.gen).to(DT[dtype])
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
        self.tables = dev(self.q_start), dev(kv_len), dev(self.table)
        self.cache = tq2.KVCache(self.k, self.v)
        self.batch = tq2.PagedBatch(*self.tables, tokens=self.tokens, max_q=max(1, *q_len), max_kv=max(kv_len))

    def slot(self, b, j):
        return int(self.table[b, j // self.page]), j % self.page

    def queries(self, heads, sharp=1.0, kind="rows"):
        x = layout((self.tokens, heads, self.dim), kind, self.dtype, self.gen)
        return x.mul_(sharp) if kind == "rows" else x


def attention_tol(step, want, weight, spread, out):
    n = max(1, max(step.kv_len))
    # (of the finite values: a key that must not be seen is not counted)
    vmax = float(np.nanmax(np.where(np.isfinite(host(step.v)), np.abs(host(step.v)), 0), initial=1.0))
    w = half_step(step.dtype)
    if out == "f32":
        w = w * w
    rel = w + 2 * (np.nan_to_num(spread, posinf=0)[..., None] * (step.dim + 8) * 2.0 ** -24) * 2 + 2.0 ** -20 + n * 2.0 ** -23
    return (half_step(out) * np.abs(want) * (1 + 2.0 ** -7) + rel * weight
            + (n * 2.0 ** -25 * vmax if step.dtype == "f16" else 0) + tiny(out))


def attend(tq2, step, heads, out="f16", window=0, causal=True, sharp=1.0, kind="rows", scale=None, workspace=True):
    q = step.queries(heads, sharp, kind)
    o = layout((step.tokens, heads, step.dim), kind, out)
    ws = tq2.attention_paged_workspace(q, step.cache, step.batch) if workspace else None
    tq2.attention_paged(q, step.cache, step.batch, out=o, window=window, causal=causal, scale=scale, workspace=ws)
    want, weight, spread = paged.attention(host(q), host(step.k), host(step.v), step.q_start, step.kv_len, step.table,
                                           step.dim ** -0.5 if scale is None else scale, window, causal)
    used = int(step.q_start[-1])
    check(o[:used], want[:used], attention_tol(step, want, weight, spread, out)[:used])
    if step.tokens > used:
        assert torch.isnan(o[used:]).all(), "a padding token was written"
    return q, o


DECODE = [
    # kv lengths, heads, kv heads, dim, page, order
    ([1], 1, 1, 8, 1, "slots"),
    ([0], 2, 1, 64, 16, "slots"),
    ([301], 32, 8, 128, 16, "slots"),
    ([5, 0, 64, 63, 65, 1, 128], 8, 2, 64, 16, "heads"),
    ([1000, 17, 2049], 8, 1, 128, 64, "heads"),
    ([700, 33], 7, 1, 80, 48, "slots"),
    ([513], 5, 5, 40, 3, "slots"),
    ([129, 511], 12, 1, 128, 100, "heads"),
    ([300, 40], 16, 1, 64, 7, "slots"),
    ([90], 24, 1, 72, 128, "slots"),
    ([260, 30], 40, 1, 128, 256, "heads"),
    ([4097, 2], 4, 2, 112, 32, "slots"),
]


@pytest.mark.parametrize("case", DECODE, ids=str)
@pytest.mark.parametrize("types", [("f16", "f16"), ("bf16", "bf16"), ("f16", "f32"), ("bf16", "f32")], ids=str)
def test_decode(tq2, case, types):
    kv_len, heads, kv_heads, dim, page, order = case
    step = Step(tq2, [1] * len(kv_len), kv_len, kv_heads, dim, page, order, types[0], seed=len(kv_len) + dim)
    attend(tq2, step, heads, types[1], sharp=2.0)


CHUNK = [
    # new tokens, kv lengths, heads, kv heads, dim, page, order
    ([2], [2], 1, 1, 64, 16, "slots"),
    ([5, 5, 5], [5, 70, 300], 14, 2, 64, 48, "slots"),
    ([3, 0, 1, 9], [128, 50, 129, 9], 8, 2, 128, 16, "heads"),
    ([17], [17], 4, 1, 128, 16, "slots"),
    ([127, 1], [127, 400], 4, 4, 128, 32, "slots"),
    ([128], [256], 2, 1, 64, 128, "heads"),
    ([129, 40], [300, 41], 3, 1, 72, 1, "slots"),
    ([200], [130], 2, 2, 128, 16, "slots"),          # the first tokens see no key
    ([300], [300], 8, 1, 128, 64, "heads"),
    ([70, 33, 260], [1000, 33, 261], 4, 1, 40, 5, "slots"),
    ([10], [2100], 12, 2, 96, 100, "heads"),
    ([6], [0], 4, 2, 64, 16, "slots"),
    ([4, 2], [0, 700], 4, 1, 8, 24, "slots"),
    ([260], [1500], 16, 2, 128, 16, "slots"),
]


@pytest.mark.parametrize("case", CHUNK, ids=str)
@pytest.mark.parametrize("types", [("f16", "f16"), ("bf16", "bf16"), ("f16", "f32"), ("bf16", "f32")], ids=str)
def test_chunk(tq2, case, types):
    q_len, kv_len, heads, kv_heads, dim, page, order = case
    step = Step(tq2, q_len, kv_len, kv_heads, dim, page, order, types[0], seed=sum(q_len) + dim)
    attend(tq2, step, heads, types[1], sharp=2.0)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [0, 1, 2, 17, 128, 129, 100_000])
@pytest.mark.parametrize("case", [([1, 1, 1], [400, 3, 129]), ([6, 3], [500, 3]), ([150, 40], [150, 333])], ids=str)
def test_masks(tq2, case, window, causal):
    step = Step(tq2, *case, 2, 64, 16, seed=window % 1000 + 3)
    attend(tq2, step, 8, "f16", window, causal)


@pytest.mark.parametrize("kind", ["heads", "slice"])
@pytest.mark.parametrize("q_len", [1, 30])
def test_strided_views_and_padding(tq2, kind, q_len):
    step = Step(tq2, [q_len, q_len], [222, 77], 2, 64, 16, dtype="bf16", pad=5)
    attend(tq2, step, 6, "bf16", kind=kind)


@pytest.mark.parametrize("q_len", [1, 40])
def test_sharp_scores_and_scale(tq2, q_len):
    # weights that fall on one key, growing and falling maxima, a negative scale
    for sharp, scale in ((40.0, None), (1.0, -0.5), (1.0, 0.0)):
        attend(tq2, Step(tq2, [q_len], [900], 1, 128, 16, seed=9), 4, "f16", sharp=sharp, scale=scale)


@pytest.mark.parametrize("rest", [float("nan"), float("inf"), -float("inf"), 65504.0])
@pytest.mark.parametrize("shape", [([1, 1], [3, 70]), ([5, 2], [5, 131]), ([50], [300])], ids=str)
def test_what_lies_past_the_end_has_no_influence(tq2, rest, shape):
    attend(tq2, Step(tq2, *shape, 1, 64, 16, rest=rest), 4)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("plane", ["k", "v"])
@pytest.mark.parametrize("shape", [([3], [40], 0), ([5], [300], 60), ([60], [200], 0), ([140], [140], 33), ([1], [500], 100)],
                         ids=str)
def test_hidden_values_have_no_influence(tq2, shape, plane, bad):
    """A key that is not finite reaches the tokens that see it and no other."""
    q_len, kv_len, window = shape
    step = Step(tq2, q_len, kv_len, 1, 64, 16, seed=4)
    n, kv = q_len[0], kv_len[0]
    for j in {kv - 1, max(0, kv - n), kv - 1 - n // 2, max(0, kv - n - 40), 0}:
        getattr(step, plane)[(*step.slot(0, j), 0, 5 if plane == "v" else 0)] = bad
    q = step.queries(4)
    o = torch.empty((step.tokens, 4, 64), device="cuda", dtype=torch.float16)
    tq2.attention_paged(q, step.cache, step.batch, out=o, window=window)
    with np.errstate(invalid="ignore"):
        want, weight, spread = paged.attention(host(q), host(step.k), host(step.v), step.q_start, kv_len, step.table,
                                               64 ** -0.5, window)
    if plane == "k" and bad == float("inf"):
        # +inf or -inf scores: only the tokens that see none of them are compared
        seen = ~np.isfinite(spread)
        keep = ~seen.any(-1)
        check(o[torch.from_numpy(keep)], want[keep], attention_tol(step, want, weight, spread, "f16")[keep])
        return
    check(o, want, attention_tol(step, want, np.nan_to_num(weight, posinf=0), spread, "f16"))


def test_long_contexts_are_split_and_joined(tq2):
    for q_len, kv_len, heads in (([1], [20_011], 8), ([4, 4], [9000, 77], 8), ([33], [7000], 4)):
        for dtype, out in (("f16", "f32"), ("bf16", "bf16")):
            step = Step(tq2, q_len, kv_len, 1, 64, 16, dtype=dtype, seed=8)
            q, o = attend(tq2, step, heads, out, sharp=2.0)
            _, again = attend_again(tq2, step, q, o)
            assert torch.equal(again, o), "another run gives other bits"


@pytest.mark.parametrize("new,heads", [(8, 1), (3, 3), (16, 1), (17, 1), (3, 8), (5, 5), (4, 8), (11, 3)], ids=str)
@pytest.mark.parametrize("dim", [64, 48, 128])
@pytest.mark.parametrize("types", [("f16", "f16"), ("bf16", "f32")], ids=str)
def test_row_counts_about_the_kernels_limits(tq2, new, heads, dim, types):
    for kv_len, window in (([40, new, 700], 0), ([3000, 5, 64], 150)):
        step = Step(tq2, [new] * 3, kv_len, 1, dim, 16, dtype=types[0], seed=new + heads)
        attend(tq2, step, heads, types[1], window, sharp=2.0)


# more items than SMs, so that CTAs go on from one to the next: short and long, one tile and two, without keys, of no token
MANY = [
    # new tokens, kv lengths, heads, kv heads, dim, window
    ([70, 1, 0, 129, 33, 300] * 7, [70, 500, 9, 129, 40, 700] * 7, 8, 8, 64, 0),
    ([300, 40] * 12, [100, 390] * 12, 24, 8, 128, 0),    # three heads a group, tokens that see no key
    ([65] * 70, [64 + i % 90 for i in range(70)], 16, 4, 40, 50),
    ([1100, 5, 900], [1100, 5, 1500], 40, 10, 64, 0),
]


@pytest.mark.parametrize("case", MANY, ids=lambda c: f"{len(c[0])}x{c[3]}x{c[4]}")
@pytest.mark.parametrize("types", [("f16", "f16"), ("bf16", "f32")], ids=str)
def test_more_items_than_sms(tq2, case, types):
    q_len, kv_len, heads, kv_heads, dim, window = case
    step = Step(tq2, q_len, kv_len, kv_heads, dim, 16, dtype=types[0], seed=dim)
    q, o = attend(tq2, step, heads, types[1], window, sharp=2.0)
    again = torch.empty_like(o)
    for _ in range(5):
        again.fill_(float("nan"))
        tq2.attention_paged(q, step.cache, step.batch, out=again, window=window)
        assert torch.equal(again, o), "another run gives other bits"


@pytest.mark.parametrize("limit_ns", [0, 20_000])
def test_waits_that_run_out_between_items(tq2, limit_ns):
    step = Step(tq2, [260, 70, 300] * 20, [700, 70, 5000] * 20, 4, 64, 16)
    q = step.queries(12)
    good = tq2.attention_paged(q, step.cache, step.batch)
    torch.cuda.synchronize()
    limit = tq2.tq2_set_wait_timeout_ns(limit_ns)
    try:
        for _ in range(3):
            tq2.attention_paged(q, step.cache, step.batch)
        assert tq2.tq2_device_status() in (tq2.TQ2_ERR_TIMEOUT, tq2.TQ2_OK)  # (a wait may find its phase in time)
    finally:
        tq2.tq2_set_wait_timeout_ns(limit)
    again = tq2.attention_paged(q, step.cache, step.batch)
    assert tq2.tq2_device_status() == tq2.TQ2_OK
    assert torch.equal(again, good)


def attend_again(tq2, step, q, o):
    """The same call with a temporary instead of a workspace."""
    again = torch.empty_like(o)
    tq2.attention_paged(q, step.cache, step.batch, out=again)
    return q, again


@pytest.mark.parametrize("q_len", [1, 20])
def test_offsets_past_32_bits(tq2, q_len):
    pages, page, heads, dim = 270_000, 16, 8, 128      # 4.4e9 elements a plane
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB")
    k, v = (torch.empty((pages, page, heads, dim), device="cuda", dtype=torch.bfloat16) for _ in range(2))
    ids = [pages - 1, 0, 131_080, pages - 2, 262_150]
    kv = 16 * len(ids) - 3
    gen = torch.Generator(device="cuda").manual_seed(1)
    new_k, new_v = (torch.randn((kv, heads, dim), device="cuda", generator=gen) for _ in range(2))
    dev = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    cache = tq2.KVCache(k, v)
    fill = tq2.PagedBatch(dev([0, kv]), dev([kv]), dev([ids]), tokens=kv, max_q=kv, max_kv=kv)
    tq2.kv_append(new_k, new_v, cache, fill)
    for i, p in enumerate(ids):
        n = min(16, kv - 16 * i)
        assert torch.equal(k[p, :n], new_k[16 * i:16 * i + n].bfloat16())
        assert torch.equal(v[p, :n], new_v[16 * i:16 * i + n].bfloat16())
    step = tq2.PagedBatch(dev([0, q_len]), dev([kv]), dev([ids]), tokens=q_len, max_q=q_len, max_kv=kv)
    q = torch.randn((q_len, 32, dim), device="cuda", generator=gen).bfloat16()
    o = tq2.attention_paged(q, cache, step)
    want, weight, spread = paged.attention(host(q), host(k[ids]), host(v[ids]), [0, q_len], [kv],
                                           [list(range(len(ids)))], dim ** -0.5)
    like = Step.__new__(Step)
    like.kv_len, like.dtype, like.dim, like.v = [kv], "bf16", dim, v[ids]
    check(o, want, attention_tol(like, want, weight, spread, "bf16"))


# ---------------------------------------------------------------------------
# append


APPEND = [
    # new tokens, kv lengths, heads (0: no q), kv heads, dim, page, order, axes, pairs, interleaved
    ([1], [1], 0, 1, 8, 1, "slots", 1, 4, False),
    ([1, 1, 1], [1, 16, 17], 8, 2, 64, 16, "slots", 1, 32, False),
    ([5, 0, 30], [5, 9, 100], 4, 4, 128, 16, "heads", 3, 64, True),
    ([40], [333], 6, 3, 80, 7, "slots", 2, 33, False),
    ([9, 3], [4, 3], 2, 1, 64, 5, "heads", 1, 32, True),      # tokens before the first key are not stored
    ([200, 1], [200, 64], 32, 8, 128, 64, "slots", 1, 0, False),
]


@pytest.mark.parametrize("case", APPEND, ids=str)
@pytest.mark.parametrize("io", [("f32", "f16"), ("f32", "bf16"), ("bf16", "bf16"), ("f16", "bf16")], ids=str)
@pytest.mark.parametrize("kind", ["rows", "slice", "heads"])
def test_append(tq2, case, io, kind):
    q_len, kv_len, heads, kv_heads, dim, page, order, axes, pairs, interleaved = case
    step = Step(tq2, q_len, kv_len, kv_heads, dim, page, order, io[1], seed=dim, rest=3.0, pad=2)
    rng = np.random.default_rng(11)
    f, axis = frequencies(pairs, axes, rng, False)
    n = step.tokens
    k, v = (layout((n, kv_heads, dim), kind, io[0], step.gen) for _ in range(2))
    q = layout((n, heads, dim), kind, io[0], step.gen) if heads else None
    where = np.full((n, 1), 0)
    for t, _, j in paged.places(step.q_start, kv_len):
        where[t] = j
    pos = where if axes == 1 else rng.integers(0, 3000, (n, axes))
    rope = tq2.Rope(f, axis if axes > 1 else None, axes=axes, interleaved=interleaved)
    before = host(step.k), host(step.v)
    q_out = layout((n, heads, dim), kind, io[1]) if heads else None
    tq2.kv_append(k, v, step.cache, step.batch, rope=rope, q=q, q_out=q_out,
                  positions=None if axes == 1 else torch.from_numpy(pos).cuda())
    used = int(step.q_start[-1])
    turned = paged.rotate(host(k), pos, f, axis, interleaved)
    want = paged.append(before[0], turned, step.q_start, kv_len, step.table)
    tol = paged.append(np.zeros(before[0].shape), rope_tol(host(k), pairs, interleaved, turned, io[1]), step.q_start,
                       kv_len, step.table)
    check(step.k, want, tol + 1e-300)          # untouched slots keep their bits
    want = paged.append(before[1], host(v.to(DT[io[1]])), step.q_start, kv_len, step.table)
    assert np.array_equal(host(step.v), want)
    if heads:
        want = paged.rotate(host(q), pos, f, axis, interleaved)
        check(q_out[:used], want[:used], rope_tol(host(q), pairs, interleaved, want, io[1])[:used])
        assert torch.isnan(q_out[used:]).all(), "a padding token was written"


def test_append_without_rope_and_in_place_queries(tq2):
    step = Step(tq2, [3, 2], [20, 2], 2, 64, 16, dtype="bf16", rest=0.0)
    q = step.queries(4)
    k, v = (step.queries(2) for _ in range(2))
    before = q.clone()
    tq2.kv_append(k, v, step.cache, step.batch, q=q, q_out=q)
    assert torch.equal(q, before)
    assert np.array_equal(host(step.k)[step.slot(0, 17)], host(k)[0])
    assert np.array_equal(host(step.v)[step.slot(1, 1)], host(v)[4])


# ---------------------------------------------------------------------------
# streams, graphs, guard bands, bad tables


@pytest.mark.parametrize("q_len", [1, 24])
def test_another_stream_and_a_captured_step(tq2, q_len):
    """Append and attention on a stream of their own, captured; a replay reads the tables' new values."""
    step = Step(tq2, [q_len] * 3, [300, 64, 25], 2, 64, 16, rest=0.0)
    page_room = tq2.PagedBatch(*step.tables, tokens=step.tokens, max_q=q_len, max_kv=step.table.shape[1] * 16)
    f, axis = frequencies(32, 1, None, False)
    rope = tq2.Rope(f)
    q, k, v = (torch.randn((step.tokens, h, 64), device="cuda", generator=step.gen).half() for h in (8, 2, 2))
    q_out, out = torch.empty_like(q), torch.empty_like(q)
    ws = tq2.attention_paged_workspace(q, step.cache, page_room)

    def one():
        tq2.kv_append(k, v, step.cache, page_room, rope=rope, q=q, q_out=q_out)
        tq2.attention_paged(q_out, step.cache, page_room, out=out, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        one()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        one()
    for shift in (0, 3, 40):
        kv_len = [300 - shift, 64 - shift // 2, 25]
        step.tables[1].copy_(torch.tensor(kv_len, dtype=torch.int32))
        q.copy_(torch.randn(q.shape, device="cuda", generator=step.gen))
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        want, weight, spread = paged.attention(host(q_out), host(step.k), host(step.v), step.q_start, kv_len,
                                               step.table, 0.125)
        check(out, want, attention_tol(step, want, weight, spread, "f16"))
        pos = np.array([[j] for _, _, j in paged.places(step.q_start, kv_len)])
        turned = paged.rotate(host(q), pos, f, axis)
        check(q_out, turned, rope_tol(host(q), 32, False, turned, "f16"))


@pytest.mark.parametrize("q_len,kv", [(1, 5), (1, 3000), (7, 40), (60, 700)])
@pytest.mark.parametrize("dim", [40, 128])
def test_guard_bands(tq2, q_len, kv, dim):
    step = Step(tq2, [q_len], [kv], 1, dim, 16)
    q = step.queries(4)
    n = q.numel()
    band = 512
    for dtype in (torch.float16, torch.float32):
        buf = torch.full((n + 2 * band,), 7.0, device="cuda", dtype=dtype)
        need = tq2.tq2_attention_paged_workspace_bytes(4, step.cache.packed, step.batch.packed)
        ws = torch.full((need + 512,), 0xA5, device="cuda", dtype=torch.uint8)
        tq2.attention_paged(q, step.cache, step.batch, out=buf[band:band + n].view(q.shape), workspace=ws[256:256 + need])
        assert (buf[:band] == 7).all() and (buf[band + n:] == 7).all(), "a write landed outside the output"
        assert (ws[:256] == 0xA5).all() and (ws[256 + need:] == 0xA5).all(), "a write landed outside the workspace"
        assert (buf[band:band + n] != 7).all()


@pytest.mark.parametrize("q_len", [1, 30])
def test_bad_tables_are_reported_and_others_unharmed(tq2, q_len):
    """A page outside the cache, a length over the table's width: the status says so, the other sequence is right
    (the arithmetic that keeps every access inside is tested on the host)."""
    step = Step(tq2, [q_len, q_len], [100, 100], 2, 64, 16, rest=0.0)
    q = step.queries(4)
    good = tq2.attention_paged(q, step.cache, step.batch)
    k, v = step.queries(2), step.queries(2)
    for table, at, value in ((2, (0, 3), 1 << 20), (2, (0, 6), -1), (1, (0,), 1 << 30), (1, (0,), -5)):
        tables = [t.clone() for t in step.tables]
        tables[table][at] = value
        bad = tq2.PagedBatch(*tables, tokens=step.tokens, max_q=q_len, max_kv=step.batch.max_kv)
        out = tq2.attention_paged(q, step.cache, bad)
        assert tq2.tq2_device_status() == tq2.TQ2_ERR_BAD_BATCH
        assert torch.equal(out[q_len:], good[q_len:])
    planes = step.k.clone(), step.v.clone()
    tables = [t.clone() for t in step.tables]
    tables[2][0] = -1
    tq2.kv_append(k, v, step.cache, tq2.PagedBatch(*tables, tokens=step.tokens, max_q=q_len, max_kv=100))
    assert tq2.tq2_device_status() == tq2.TQ2_ERR_BAD_BATCH
    assert torch.equal(step.k[step.slot(1, 99)], k[-1]) and torch.equal(step.v[step.slot(1, 99)], v[-1])
    for b in range(100 // 16 + 1):   # the first sequence's pages are as they were
        p = int(step.table[0, b])
        assert torch.equal(step.k[p], planes[0][p]) and torch.equal(step.v[p], planes[1][p])
    assert tq2.tq2_device_status() == tq2.TQ2_OK


def test_operands_off_the_device_are_refused(tq2):
    step = Step(tq2, [2], [20], 1, 64, 16, rest=0.0)
    q = step.queries(2)
    H = tq2.tq2_heads
    pinned = torch.zeros(1 << 16, dtype=torch.float16).pin_memory()
    at = (pinned.data_ptr() + 255) & ~255
    here, there = H(q.data_ptr(), 2, 128, 64, 1), H(at, 2, 128, 64, 1)
    one = H(at, 1, 64, 64, 1), H(q.data_ptr(), 1, 64, 64, 1)
    f, _ = frequencies(32, 1, None, False)
    rope = tq2.Rope(f)
    pos = torch.zeros(2, dtype=torch.int64, device="cuda")
    L, bad = tq2.lib, tq2.TQ2_ERR_INVALID_ARG
    assert L.tq2_rope_axes(there, here, None, None, None, None, pos.data_ptr(), rope.packed, 2, 64, 0, None) == bad
    assert L.tq2_rope_axes(here, here, None, None, None, None, at, rope.packed, 2, 64, 0, None) == bad
    assert L.tq2_kv_append(None, None, *one, None, None, step.batch.packed, step.cache.packed, None) == bad
    assert L.tq2_attention_paged(there, here, step.cache.packed, step.batch.packed, 0.1, 0, 1, None, 0, None) == bad
    off = tq2.tq2_batch(step.tables[0], at, step.tables[2], 1, 2, 2, 20, step.table.shape[1])
    assert L.tq2_attention_paged(here, H(step.queries(2).data_ptr(), 2, 128, 64, 1), step.cache.packed, off, 0.1, 0, 1,
                                 None, 0, None) == bad


# ---------------------------------------------------------------------------
# waits that give up, and the operators together


@pytest.mark.parametrize("q_len,kv", [(1, 3000), (4, 100), (70, 900), (300, 300), (40, 9000)])
def test_a_wait_that_runs_out_is_reported_and_the_context_goes_on(tq2, q_len, kv):
    step = Step(tq2, [q_len, q_len], [kv, kv // 2 + 1], 2, 128, 16)
    q = step.queries(6)
    good = tq2.attention_paged(q, step.cache, step.batch)
    torch.cuda.synchronize()
    limit = tq2.tq2_set_wait_timeout_ns(0)
    try:
        for _ in range(3):
            tq2.attention_paged(q, step.cache, step.batch)
        assert tq2.tq2_device_status() in (tq2.TQ2_ERR_TIMEOUT, tq2.TQ2_OK)  # (a wait may find its phase in time)
    finally:
        tq2.tq2_set_wait_timeout_ns(limit)
    again = tq2.attention_paged(q, step.cache, step.batch)
    assert tq2.tq2_device_status() == tq2.TQ2_OK
    assert torch.equal(again, good)


def test_a_decoder_of_ternary_layers(tq2):
    """Prompts in chunks and decoding by graph replays give the logits of one pass over everything."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "ternary_decoder.py")
    spec = importlib.util.spec_from_file_location("ternary_decoder", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    model = ex.Decoder(layers=2, ffn=512, vocab=256)
    rng = np.random.default_rng(0)
    prompts = [rng.integers(0, 256, n).tolist() for n in (70, 5, 33)]
    tokens, _ = ex.generate(model, prompts, 6, chunk=32)
    tokens = tokens.tolist()
    # each sequence alone, prompt and continuation in one step: the token after each position is the same, but where
    # the two best logits are nearer than the activations' binary16 and the cache's bf16 roundings move them
    for p, row in zip(prompts, tokens):
        text = p + row
        seqs = ex.Sequences(1, len(text))
        logits = model.step(torch.tensor(text, device="cuda"), model.new_caches(seqs.pages), seqs.batch([len(text)]))
        for i, got in enumerate(row):
            at = logits[len(p) - 1 + i].double()
            assert at.max() - at[got] <= 0.05 * at.std(), (len(p), i)
    assert torch.isfinite(ex.joint_tokens(torch.randn(77 + 64, 3 * 4 * 64, device="cuda"), 4, 64, 77, 8)).all()

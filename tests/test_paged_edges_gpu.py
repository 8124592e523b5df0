"""GPU tests of the paged operators where calls go wrong or nearly so: waits that run out, tables that contradict one
another, weights near the end of a type's range, layouts that interleave.  Tolerances as in test_paged_gpu.py; where a
test needs a tighter one, its derivation stands beside it."""

import numpy as np
import pytest

from oracle import paged
from test_paged_edges import KEPT, telling_scores
from test_paged_gpu import DT, Step, attention_tol, check, frequencies, half_step, host, rope_tol

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tq2():
    import dit_tq2_g128_gb300 as m
    return m


@pytest.fixture(autouse=True)
def status_is_clean(tq2):
    yield
    assert tq2.tq2_device_status() == tq2.TQ2_OK


class Limit:
    """A limit on the device's waits, put back at the end."""

    def __init__(self, tq2, ns):
        self.tq2, self.ns = tq2, ns

    def __enter__(self):
        torch.cuda.synchronize()
        self.before = self.tq2.tq2_set_wait_timeout_ns(self.ns)

    def __exit__(self, *_):
        self.tq2.tq2_set_wait_timeout_ns(self.before)


@pytest.mark.parametrize("kv", [40, 100, 190])
def test_copies_land_before_a_cta_that_gave_up_is_gone(tq2, kv):
    """Runs of one to three tiles, whose producer never waits: what they copied must not land in the shared memory of
    the CTAs that come next."""
    few = Step(tq2, [4] * 40, [kv] * 40, 8, 128, 16)
    many = Step(tq2, [130, 40], [200, 90], 4, 128, 16, seed=1)
    q, r = few.queries(16), many.queries(4)
    good, next_good = tq2.attention_paged(q, few.cache, few.batch), tq2.attention_paged(r, many.cache, many.batch)
    for _ in range(20):
        with Limit(tq2, 0):
            for _ in range(3):
                tq2.attention_paged(q, few.cache, few.batch)
        assert torch.equal(tq2.attention_paged(r, many.cache, many.batch), next_good)
        assert torch.equal(tq2.attention_paged(q, few.cache, few.batch), good)
    tq2.tq2_device_status()


def test_sequences_that_claim_the_same_tokens(tq2):
    """Fifty of a hundred sequences claim the same 3000 tokens over 2^30 keys each: more work than 32 bits count."""
    ints = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    k = torch.zeros((1, 1 << 20, 1, 8), device="cuda", dtype=torch.float16)
    q = torch.ones((3000, 1, 8), device="cuda", dtype=torch.float16)
    table = torch.zeros((100, 1 << 10), dtype=torch.int32, device="cuda")
    batch = tq2.PagedBatch(ints(*([0, 3000] * 50 + [0])), ints(*[1 << 30] * 100), table, tokens=3000, max_q=3000, max_kv=1 << 30)
    tq2.attention_paged(q, tq2.KVCache(k, k.clone()), batch)
    assert tq2.tq2_device_status() == tq2.TQ2_ERR_BAD_BATCH


@pytest.mark.parametrize("what", ["more keys than max_kv", "more keys than the table", "more tokens than max_q"])
def test_append_of_a_bad_batch_stores_nothing_of_its_sequence(tq2, what):
    step = Step(tq2, [2, 3, 1], [48, 40, 17], 2, 64, 16, rest=0.0)
    k, v = step.queries(2), step.queries(2)
    tables, max_q, max_kv, bad = [t.clone() for t in step.tables], 3, 48, 0
    if what == "more keys than max_kv":
        tables[1][0] = 49
    elif what == "more keys than the table":
        tables[1][0], max_kv = 60, 1000
    else:
        max_q, bad = 2, 1
    want = [step.k.clone(), step.v.clone()]
    for b in range(3):
        for i in range(step.q_len[b]):
            if b != bad:
                at = step.slot(b, step.kv_len[b] - step.q_len[b] + i)
                for plane, x in zip(want, (k, v)):
                    plane[at] = x[int(step.q_start[b]) + i]
    batch = tq2.PagedBatch(*tables, tokens=step.tokens, max_q=max_q, max_kv=max_kv)
    tq2.kv_append(k, v, step.cache, batch)
    assert tq2.tq2_device_status() == tq2.TQ2_ERR_BAD_BATCH
    assert torch.equal(step.k, want[0]) and torch.equal(step.v, want[1])


@pytest.mark.parametrize("q_len", [1, 6, 40, 300])
@pytest.mark.parametrize("entry", [-1, 1 << 20])
def test_a_page_outside_the_cache_reads_as_zeros(tq2, q_len, entry):
    step = Step(tq2, [q_len, q_len], [310, 300], 2, 64, 16)
    q = step.queries(4)
    tables = [t.clone() for t in step.tables]
    tables[2][0, 3] = entry
    tables[2][0, 19] = entry
    out = tq2.attention_paged(q, step.cache, tq2.PagedBatch(*tables, tokens=step.tokens, max_q=q_len, max_kv=310))
    assert tq2.tq2_device_status() == tq2.TQ2_ERR_BAD_BATCH
    pages = step.k.shape[0]
    k, v = (np.concatenate([host(p), np.zeros((1, *p.shape[1:]))]) for p in (step.k, step.v))
    table = step.table.copy()
    table[0, [3, 19]] = pages
    want, weight, spread = paged.attention(host(q), k, v, step.q_start, step.kv_len, table, 0.125)
    check(out, want, attention_tol(step, want, weight, spread, "f16"))


@pytest.mark.parametrize("q_len", [1, 4, 40, 300])
@pytest.mark.parametrize("out", ["f16", "f32"])
@pytest.mark.parametrize("low", [9.0, 11.0, 13.3984375])
def test_small_weights_beside_large_ones(tq2, q_len, out, low):
    """Every 16th key has weight 1 and v = 0, the others e^-low (down to 2^-19) and v = 1000: the result is theirs alone.
    Weights keep half a step of binary16 (f32 outputs: its square, 2^-22), or 2^-32 of the largest; scores up to 20 in log2
    units leave the exponential 2^-19."""
    step = Step(tq2, [q_len], [400], 1, 64, 16, rest=0.0)
    j = torch.arange(400, device="cuda")
    p, o = torch.from_numpy(step.table[0].astype(np.int64)).cuda()[j // 16], j % 16
    step.k.zero_()
    step.v.zero_()
    large = (j % 16 == 0)
    step.k[p, o, 0, 0] = torch.where(large, low, 0.0).half()
    step.v[p, o, 0, :] = torch.where(large, 0.0, 1000.0).half()[:, None]
    q = torch.zeros((q_len, 4, 64), device="cuda", dtype=torch.float16)
    q[..., 0] = 1
    got = torch.empty(q.shape, device="cuda", dtype=DT[out])
    tq2.attention_paged(q, step.cache, step.batch, out=got, scale=1.0, causal=False)
    want, weight, _ = paged.attention(host(q), host(step.k), host(step.v), [0, q_len], [400], step.table, 1.0, causal=False)
    w = 2.0 ** -11 if out == "f16" else 2.0 ** -22
    check(got, want, half_step(out) * np.abs(want) + (w + 2.0 ** -19) * weight + 400 * 2.0 ** -32 * 1000)


def test_interleaved_projection_in_place(tq2):
    gen = torch.Generator(device="cuda").manual_seed(5)
    f, _ = frequencies(64, 1, np.random.default_rng(5), False)
    fused = torch.randn((9, 4, 3, 128), device="cuda", generator=gen)
    before = host(fused)
    pos = np.arange(9).reshape(9, 1) * 7
    rope, at = tq2.Rope(f), torch.from_numpy(pos).cuda()
    tq2.rope_axes(fused[:, :, 0], fused[:, :, 1], positions=at, rope=rope, out=(fused[:, :, 0], fused[:, :, 1]))
    for i, turned in enumerate((True, True, False)):
        want = paged.rotate(before[:, :, i], pos, f if turned else [], [0] * 64)
        check(fused[:, :, i], want, rope_tol(before[:, :, i], 64 if turned else 0, False, want, "f32"), str(i))


def test_a_long_item_is_not_a_wait_that_ran_out(tq2):
    """152 whole items of 800 blocks each take a millisecond, each block little more than one microsecond."""
    step = Step(tq2, [1216], [102_400], 8, 64, 64)
    q = step.queries(32)
    good = tq2.attention_paged(q, step.cache, step.batch)
    with Limit(tq2, 100_000):
        got = tq2.attention_paged(q, step.cache, step.batch)
        assert tq2.tq2_device_status() == tq2.TQ2_OK
    assert torch.equal(got, good)


def long_items(tq2):
    """Whole items of up to 40 blocks: the next one is claimed near the end, which no limit of 0 waits for."""
    return Step(tq2, [260, 70, 300] * 20, [1700, 70, 5000] * 20, 4, 64, 16)


def test_a_wait_that_cannot_be_met_is_reported(tq2):
    step = long_items(tq2)
    q = step.queries(12)
    good = tq2.attention_paged(q, step.cache, step.batch)
    for _ in range(5):
        with Limit(tq2, 0):
            tq2.attention_paged(q, step.cache, step.batch)
            assert tq2.tq2_device_status() == tq2.TQ2_ERR_TIMEOUT
        assert torch.equal(tq2.attention_paged(q, step.cache, step.batch), good)


def test_a_wait_of_few_rows_that_runs_out_is_reported(tq2):
    """The first of 24 tiles, where some rows see a key and others do not, holds nothing but infinities, which the
    consumers hand to the rows one by one for half a millisecond; the copies of the fourth tile wait for them."""
    step = Step(tq2, [32], [2000], 1, 64, 16)
    j = torch.arange(512, device="cuda")
    p, o = torch.from_numpy(step.table[0].astype(np.int64)).cuda()[j // 16], j % 16
    q = step.queries(1)
    step.v[p, o] = float("inf")
    good = tq2.attention_paged(q, step.cache, step.batch, window=1500)
    torch.cuda.synchronize()
    for _ in range(5):
        with Limit(tq2, 0):
            tq2.attention_paged(q, step.cache, step.batch, window=1500)
            assert tq2.tq2_device_status() == tq2.TQ2_ERR_TIMEOUT
        assert torch.equal(tq2.attention_paged(q, step.cache, step.batch, window=1500).view(torch.int16), good.view(torch.int16))


def test_the_status_reports_both_kinds_one_after_the_other(tq2):
    step = long_items(tq2)
    q = step.queries(12)
    tables = [t.clone() for t in step.tables]
    tables[1][0] = -1
    bad = tq2.PagedBatch(*tables, tokens=step.tokens, max_q=300, max_kv=5000)
    with Limit(tq2, 0):
        tq2.attention_paged(q, step.cache, bad)
        assert tq2.tq2_device_status() == tq2.TQ2_ERR_TIMEOUT
    assert tq2.tq2_device_status() == tq2.TQ2_ERR_BAD_BATCH
    assert tq2.tq2_device_status() == tq2.TQ2_OK


def pool_stream(t):
    for seg in torch.cuda.memory_snapshot():
        if seg["address"] <= t.data_ptr() < seg["address"] + seg["total_size"]:
            return seg["stream"]


@pytest.mark.parametrize("as_int", [False, True])
def test_results_belong_to_the_stream_that_writes_them(tq2, as_int):
    step = Step(tq2, [3], [40], 2, 64, 16, rest=0.0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s = side.cuda_stream if as_int else side
    q, k, v = step.queries(4), step.queries(2), step.queries(2)
    rope = tq2.Rope([1.0, 0.1])
    w = torch.zeros(tq2.tq2_soa_bytes(64, 128), dtype=torch.uint8, device="cuda")
    x = torch.zeros((2, 128), device="cuda")
    torch.cuda.synchronize()
    got = [tq2.attention_paged(q, step.cache, step.batch, stream=s),
           tq2.kv_append(k, v, step.cache, step.batch, q=q, stream=s),
           *tq2.rope_axes(q, k, v, positions=torch.arange(3, device="cuda"), rope=rope, stream=s),
           tq2.matmul(w, x, n=64, k=128, stream=s)]
    side.synchronize()
    assert [pool_stream(t) for t in got] == [side.cuda_stream] * len(got)


def test_results_of_the_default_stream_by_its_handle(tq2):
    step = Step(tq2, [3], [40], 2, 64, 16, rest=0.0)
    q = step.queries(4)
    with torch.cuda.stream(torch.cuda.Stream()):
        got = tq2.attention_paged(q, step.cache, step.batch, stream=0)
    torch.cuda.synchronize()
    assert pool_stream(got) == 0


def test_an_uploaded_weight_belongs_to_its_stream(tq2):
    w = np.random.default_rng(0).integers(0, 256, tq2.tq2_soa_bytes(64, 128), dtype=np.uint8)
    want = tq2.upload_weight(w, 64, 128)
    side = torch.cuda.Stream()
    got = tq2.upload_weight(w, 64, 128, stream=side)
    side.synchronize()
    assert torch.equal(got, want) and pool_stream(got) == side.cuda_stream


def test_first_columns_of_a_wider_table(tq2):
    step = Step(tq2, [2, 3, 1], [30, 40, 17], 2, 64, 16, rest=0.0)
    q = step.queries(4)
    good = tq2.attention_paged(q, step.cache, step.batch)
    wide = torch.full((3, 9), -1, dtype=torch.int32, device="cuda")
    wide[:, :3] = step.tables[2]
    got = tq2.attention_paged(q, step.cache, tq2.PagedBatch(*step.tables[:2], wide[:, :3], tokens=6, max_q=3, max_kv=40))
    assert torch.equal(got, good)
    with pytest.raises(ValueError):
        tq2.PagedBatch(*step.tables[:2], wide[:, 6:], tokens=6, max_q=3, max_kv=40)
    # one sequence, one entry: strides of single elements say nothing
    one = Step(tq2, [1], [5], 2, 64, 16, rest=0.0)
    q = one.queries(2)
    tables = [t.repeat_interleave(2, -1)[..., ::2] for t in (one.tables[0], one.tables[1], one.tables[2])]
    tables[0] = one.tables[0]
    got = tq2.attention_paged(q, one.cache, tq2.PagedBatch(*tables, tokens=1, max_q=1, max_kv=5))
    assert torch.equal(got, tq2.attention_paged(q, one.cache, one.batch))


def test_positions_of_another_shape_are_refused(tq2):
    rope = tq2.Rope([1.0, 0.1], axis=[0, 1], axes=2)
    x = torch.zeros((3, 1, 4), device="cuda")
    with pytest.raises(ValueError):
        tq2.rope_axes(x, positions=torch.zeros((2, 3), dtype=torch.int64, device="cuda"), rope=rope)


COUNTS = [
    # new tokens, kv lengths, heads, kv heads, dim, page, window
    ([1], [20_011], 8, 1, 64, 16, 0),
    ([1], [131_071], 16, 2, 128, 64, 0),
    ([1] * 5, [4097, 63, 9000, 1, 513], 8, 2, 128, 48, 0),
    ([4, 4], [9000, 77], 8, 1, 64, 1, 700),
    ([1] * 70, [900 + 13 * i for i in range(70)], 4, 1, 40, 100, 0),
    ([33], [7000], 4, 1, 64, 16, 0),
    ([260, 5], [1500, 3000], 16, 2, 128, 16, 0),
    ([300], [20_000], 8, 1, 64, 20, 3000),
    ([300, 40] * 12, [900, 390] * 12, 24, 8, 128, 16, 0),
    ([64], [131_000], 8, 1, 128, 64, 0),
]


@pytest.mark.parametrize("case", COUNTS, ids=lambda c: f"{c[0][0]}x{len(c[0])}-{max(c[1])}-{c[4]}-{c[5]}-{c[6]}")
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_every_key_counts_once(tq2, case, dtype):
    """k = 0 and v = 1 in feature j % dim: every weight is the same and every sum a whole number below 2^24 times it, so a
    result is the share of the visible keys with that remainder, to the roundings of 1 / l and of the product."""
    q_len, kv_len, heads, kv_heads, dim, page, window = case
    step = Step(tq2, q_len, kv_len, kv_heads, dim, page, "slots", dtype)
    for b, n in enumerate(kv_len):
        j = torch.arange(n, device="cuda")
        p, o = torch.from_numpy(step.table[b].astype(np.int64)).cuda()[j // page], j % page
        step.k[p, o] = 0
        step.v[p, o] = torch.nn.functional.one_hot(j % dim, dim)[:, None].to(DT[dtype])
    q = step.queries(heads)
    got = torch.empty(q.shape, device="cuda")
    tq2.attention_paged(q, step.cache, step.batch, out=got, window=window)
    want = np.zeros((step.tokens, dim))
    d = np.arange(dim)
    for t, _, pos in paged.places(step.q_start, kv_len):
        lo, hi = max(0, pos + 1 - window) if window else 0, pos + 1
        if hi > lo:
            want[t] = ((hi - 1 - d) // dim - (lo - 1 - d) // dim) / (hi - lo)
    want = np.repeat(want[:, None], heads, 1)
    check(got, want, 2.0 ** -22 * want + 1e-30)


@pytest.mark.parametrize("dtype,rows", KEPT, ids=str)
@pytest.mark.parametrize("dim", [64, 128])
def test_f32_outputs_keep_the_terms_of_the_weights(tq2, dtype, rows, dim):
    """As the host's test of these scores: 64 keys of score 0 and v = 0, but every 16th of score s and v = 1."""
    s = telling_scores(dtype, rows)
    q_len = 1 if rows == "few" else 40
    step = Step(tq2, [q_len] * len(s), [64] * len(s), 1, dim, 16, "slots", dtype, rest=0.0)
    step.k.zero_()
    step.v.zero_()
    for b, x in enumerate(s):
        for j in range(3, 64, 16):
            step.k[(*step.slot(b, j), 0, 0)] = float(x)
            step.v[step.slot(b, j)] = 1.0
    q = torch.zeros((step.tokens, 4, dim), device="cuda", dtype=DT[dtype])
    q[..., 0] = 1
    got = torch.empty(q.shape, device="cuda")
    tq2.attention_paged(q, step.cache, step.batch, out=got, scale=1.0, causal=False)
    w = np.repeat(np.exp(s) / (15 + np.exp(s)), q_len)[:, None, None] + np.zeros(got.shape)
    check(got, w, KEPT[dtype, rows][1] * w)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("to", ["f32", "f16"])
def test_f32_rotations_keep_f32s_bits(tq2, interleaved, to):
    """Sines and cosines off by 1e-7, one product's rounding (2^-24) and the result's: together below 2^-22 of |a| + |b|."""
    rng = np.random.default_rng(3)
    f, _ = frequencies(64, 1, rng, False)
    pos = np.concatenate([np.arange(200), rng.integers(-(1 << 20), 1 << 20, 200)]).reshape(400, 1)
    x = torch.randn((400, 3, 128), device="cuda", generator=torch.Generator(device="cuda").manual_seed(3))
    out = torch.empty(x.shape, device="cuda", dtype=DT[to])
    tq2.rope_axes(x, positions=torch.from_numpy(pos).cuda(), rope=tq2.Rope(f, interleaved=interleaved), out=[out])
    want = paged.rotate(host(x), pos, f, [0] * 64, interleaved)
    near = np.abs(host(x)).reshape(400, 3, 64, 2) if interleaved else np.abs(host(x)).reshape(400, 3, 2, 64).swapaxes(2, 3)
    near = near.sum(-1)
    near = np.repeat(near, 2, -1) if interleaved else np.concatenate([near, near], -1)
    check(out, want, 2.0 ** -22 * near + (half_step(to) * np.abs(want) * 1.001 + 2.0 ** -25 if to == "f16" else 0))


@pytest.mark.parametrize("q_len", [1, 40])
def test_a_loose_bound_of_the_keys_is_no_size(tq2, q_len):
    """max_kv may be far above what the tables hold: 2^30 keys for each of 300 sequences would be too many to share out."""
    step = Step(tq2, [q_len] * 300, [41 + i % 50 for i in range(300)], 8, 64, 16)
    q = step.queries(8)
    good = tq2.attention_paged(q, step.cache, step.batch)
    loose = tq2.PagedBatch(*step.tables, tokens=step.tokens, max_q=q_len, max_kv=1 << 30)
    for workspace in (None, tq2.attention_paged_workspace(q, step.cache, loose)):
        assert torch.equal(tq2.attention_paged(q, step.cache, loose, workspace=workspace), good)

"""Routing and sampling on a GB300 against the 64-bit oracle."""

import numpy as np
import pytest

from oracle import decode

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def tq2():
    import dit_tq2_g128_gb300 as m
    return m


def logits_of(rng, rows, n, dtype, sharp=1.0, pad=0, lead=0):
    """A [rows, n] view with rows of n + pad elements, its first element `lead` after an aligned one; what lies between is
    larger than any logit."""
    values = torch.from_numpy(rng.standard_normal((rows, n)) * 3 * sharp - np.log(rng.uniform(1, n + 1, (rows, n))))
    base = torch.full((lead + rows * (n + pad),), 1e4, dtype=DTYPES[dtype], device="cuda")
    view = base[lead:].view(rows, n + pad)[:, :n]
    view.copy_(values)
    return view


# ---------------------------------------------------------------------------
# routing


def check_route(tq2, logits, k, sigmoid, normalize, scale):
    e, w = tq2.moe_route(logits, k, sigmoid=sigmoid, normalize=normalize, scale=scale)
    x = logits.double().cpu().numpy()
    we, ww = decode.route(x, k, sigmoid, normalize, scale)
    assert e.dtype == torch.int32 and w.dtype == torch.float32 and e.shape == w.shape == (len(x), k)
    assert np.array_equal(e.cpu().numpy(), we)
    got = w.cpu().numpy().astype(np.float64)
    fine = np.isfinite(ww)
    assert np.array_equal(np.isnan(got), np.isnan(ww))
    # exp's argument is off by 2^-24 of itself, exp by 2 steps, the sums (at most 32 + 5 of a lane and over lanes) by 37
    # half steps each, quotient and scale by one: (|d| + 64) 2^-23 of the weight; weights below 2^-126 by a step of 2^-149
    with np.errstate(all="ignore"):
        d = np.abs(np.take_along_axis(x, we.astype(np.int64), 1) - np.max(x, axis=1, keepdims=True))
    tol = (np.where(np.isfinite(d), d, 0) + 64) * 2.0 ** -23 * np.abs(np.where(fine, ww, 0)) + 2.0 ** -125
    assert np.all(np.abs(got - ww)[fine] <= tol[fine])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,n,k", [(1, 1, 1), (3, 2, 2), (1, 8, 2), (9, 31, 5), (7, 32, 32), (8, 33, 32), (17, 64, 6),
                                        (64, 65, 1), (33, 128, 8), (130, 129, 7), (70, 256, 8), (5, 511, 12),
                                        (9, 1000, 31), (3, 1024, 32)])
@pytest.mark.parametrize("sigmoid,normalize,scale", [(False, True, 1.0), (False, False, 2.5), (True, True, 2.5),
                                                     (True, False, 1.0)])
def test_route(tq2, dtype, tokens, n, k, sigmoid, normalize, scale):
    rng = np.random.default_rng(tokens * 1000 + n)
    check_route(tq2, logits_of(rng, tokens, n, dtype, pad=n % 3, lead=tokens % 2), k, sigmoid, normalize, scale)


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("normalize", [False, True])
def test_route_masked_rows_and_ties(tq2, sigmoid, normalize):
    rng = np.random.default_rng(5)
    x = rng.integers(-3, 4, (12, 70)).astype(np.float32)  # many equal logits
    x[1, :] = -INF
    x[2, 3:] = -INF                      # fewer left than are taken
    x[3, ::2] = -INF
    x[4, :] = 0.0
    x[4, 5::3] = -0.0                    # equal zeros
    x[5] = -200.0                        # sigmoids that vanish
    check_route(tq2, torch.from_numpy(x).cuda(), 6, sigmoid, normalize, 1.0)


def test_route_nan_comes_last(tq2):
    x = np.array([[1.0, NAN, 0.5, -INF, 2.0], [NAN] * 5, [0.0, 1.0, -NAN, 3.0, 2.0]], dtype=np.float32)
    e, w = tq2.moe_route(torch.from_numpy(x).cuda(), 5, sigmoid=True, normalize=False)
    assert e.tolist() == [[4, 0, 2, 3, 1], [0, 1, 2, 3, 4], [3, 4, 1, 0, 2]]
    w = w.cpu().numpy()
    assert np.array_equal(np.isnan(w), np.isnan(np.take_along_axis(x, e.cpu().numpy().astype(int), 1)))


@pytest.mark.parametrize("sigmoid", [False, True])
@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("k", [1, 2, 4])
def test_route_nan_and_infinity_go_through_the_formulas(tq2, sigmoid, normalize, k):
    """A softmax has them in its sum, chosen or not; sigmoids only where they are chosen."""
    x = np.random.default_rng(17).standard_normal((9, 40)).astype(np.float32)
    x[0, 7] = NAN
    x[1, 39] = INF
    x[2, :2] = INF
    x[3], x[3, 5] = -INF, NAN
    x[4], x[4, 38:] = -INF, (INF, NAN)
    x[5], x[5, 3] = NAN, 1.0
    x[6] = NAN
    x[7], x[7, 4:7] = -INF, NAN
    check_route(tq2, torch.from_numpy(x).cuda(), k, sigmoid, normalize, 1.5)


def test_route_given_outputs_stream_and_replay(tq2):
    rng = np.random.default_rng(6)
    x = logits_of(rng, 40, 100, "bf16")
    e, w = (torch.full((40, 4), -7, dtype=d, device="cuda") for d in (torch.int32, torch.float32))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = tq2.moe_route(x, 4, experts=e, weights=w, stream=side)
    assert got[0] is e and got[1] is w
    side.synchronize()
    want = tq2.moe_route(x, 4)
    assert torch.equal(e, want[0]) and torch.equal(w, want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tq2.moe_route(x, 4, experts=e, weights=w)
    for seed in (7, 8):
        x.copy_(logits_of(np.random.default_rng(seed), 40, 100, "bf16"))
        graph.replay()
        want = tq2.moe_route(x, 4)
        assert torch.equal(e, want[0]) and torch.equal(w, want[1])


def test_empty_calls(tq2):
    e, w = tq2.moe_route(torch.empty((0, 16), device="cuda"), 2)
    assert e.shape == w.shape == (0, 2)
    t, p = tq2.sample(torch.empty((0, 16), device="cuda"), torch.empty(0, device="cuda"))
    assert t.shape == p.shape == (0,)


def test_tensor_refusals(tq2):
    x = torch.zeros((4, 16), device="cuda")
    u = torch.zeros(4, device="cuda")
    for bad in (x.double(), x.t()[:4], x[0]):
        with pytest.raises((ValueError, tq2.TQ2Error)):
            tq2.moe_route(bad, 2)
        with pytest.raises((ValueError, tq2.TQ2Error)):
            tq2.sample(bad, u)
    with pytest.raises(tq2.TQ2Error):
        tq2.moe_route(x, 17)
    with pytest.raises(ValueError):
        tq2.moe_route(x, 2, experts=torch.zeros((4, 2), dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        tq2.sample(x, u[:3])
    with pytest.raises(ValueError):
        tq2.sample(x, u, top_k=u)
    with pytest.raises(ValueError):
        tq2.sample(x, u, top_p=u.cpu())
    with pytest.raises(tq2.TQ2Error):
        tq2.sample(torch.zeros((1, (1 << 18) + 1), device="cuda"), u[:1])
    with pytest.raises(tq2.TQ2Error):  # pinned host memory
        tq2.tq2_sample(torch.zeros((4, 16)).pin_memory(), tq2.TQ2_F32, 16, u, None, torch.zeros(4, dtype=torch.int64, device="cuda"), None, 4, 16)


# ---------------------------------------------------------------------------
# sampling


def check_sample(tq2, logits, u, temperature=None, top_k=None, top_p=None, min_p=None):
    """The drawn tokens are the oracle's, but where a border lies within what the weights are off by (2^-30, and the
    oracle's own sums' 2^-36); how many such rows there are."""
    rows = logits.shape[0]
    put = lambda v, t=torch.float32: None if v is None else torch.tensor(v, dtype=t, device="cuda")  # noqa: E731
    filters = dict(temperature=put(temperature), top_k=put(top_k, torch.int32), top_p=put(top_p), min_p=put(min_p))
    ut = put(u)
    tokens, prob = tq2.sample(logits, ut, **filters)
    assert tokens.dtype == torch.int64 and prob.dtype == torch.float32 and tokens.shape == prob.shape == (rows,)
    x, got, p = logits.double().cpu().numpy(), tokens.tolist(), prob.cpu().numpy().astype(np.float64)
    host = {k: (v.double().cpu().numpy() if v is not None else None) for k, v in filters.items()}
    uh, near = ut.double().cpu().numpy(), 0
    for r in range(rows):
        f = {k: float(v[r]) for k, v in host.items() if v is not None}
        if "top_k" in f:
            f["top_k"] = int(f["top_k"])
        want, wp, margin = decode.sample(x[r], uh[r], **f)
        if margin < 4e-9 and got[r] != want:
            near += 1
            continue
        assert got[r] == want, (r, got[r], want, uh[r], f, margin)
        # the quotient of sums each within 2^-30, rounded once (2^-24)
        assert margin < 4e-9 or abs(p[r] - wp) <= wp * 2.0 ** -23, (r, p[r], wp)
    return near


FILTERS = {
    "none": {},
    "temperature": dict(temperature=(0.3, 2.0)),
    "top_k": dict(top_k=(1, 60)),
    "top_p": dict(top_p=(0.05, 1.0)),
    "min_p": dict(min_p=(0.0, 0.5)),
    "all": dict(temperature=(0.5, 1.5), top_k=(-5, 300), top_p=(0.5, 1.1), min_p=(-0.05, 0.2)),
    "k_p": dict(top_k=(1, 2000), top_p=(0.5, 0.99)),
}


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,vocab,sharp", [(1, 1, 1), (5, 2, 1), (3, 31, 1), (40, 1000, 1), (7, 4097, 2), (3, 32_000, 1),
                                              (2, 65_537, 0.3), (33, 9_001, 0.2), (2, 131_072, 2), (1, 200_001, 1),
                                              (1, 262_144, 0.5)])
@pytest.mark.parametrize("filters", FILTERS)
def test_sample(tq2, dtype, rows, vocab, sharp, filters):
    rng = np.random.default_rng(rows + vocab)
    logits = logits_of(rng, rows, vocab, dtype, sharp, pad=vocab % 5, lead=rows % 2)
    f = {}
    for name, (lo, hi) in FILTERS[filters].items():
        v = rng.uniform(lo, hi, rows)
        f[name] = np.round(v).astype(int).tolist() if name == "top_k" else v.tolist()
    near = check_sample(tq2, logits, rng.random(rows).tolist(), **f)
    assert near <= 1 + rows // 100


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,vocab", [(200, 30_011), (150, 1025), (40, 131_000)])
def test_sample_without_top_k(tq2, dtype, rows, vocab):
    """Rows from nearly flat to nearly decided, with every mix of the other filters."""
    rng = np.random.default_rng(vocab)
    x = rng.standard_normal((rows, vocab)) * np.exp(rng.uniform(-4, 2, (rows, 1)))
    x[::5] = np.round(x[::5] * 4) / 4          # many equal
    x[1::7, vocab // 3:] = -INF
    x[2::9, :3] += 12.0                        # a few that outweigh the rest
    logits = torch.from_numpy(x).to(DTYPES[dtype]).cuda()
    f = dict(temperature=np.exp(rng.uniform(-1, 1, rows)).tolist(),
             top_p=np.where(rng.random(rows) < 0.7, 1 - rng.uniform(0, 1, rows) ** 3, 1.0).tolist(),
             min_p=np.where(rng.random(rows) < 0.3, rng.uniform(0, 0.05, rows), 0.0).tolist())
    near = check_sample(tq2, logits, rng.random(rows).tolist(), **f)
    assert near <= 1 + rows // 100


@pytest.mark.parametrize("vocab", [5, 1003, 70_000])
def test_every_token_by_its_share(tq2, vocab):
    """u steps through the whole order: equal weights' tokens come in the order of their indices."""
    rows = 64
    u = [(r + 0.5) / rows for r in range(rows)]
    x = torch.zeros((rows, vocab), device="cuda")
    tokens, prob = tq2.sample(x, torch.tensor(u, device="cuda"))
    assert tokens.tolist() == [int(np.float64(np.float32(a)) * vocab) for a in u]
    assert np.allclose(prob.cpu().numpy(), 1 / vocab, rtol=2.0 ** -23)
    x[:, ::2] = -1.0  # two levels, both large
    check_sample(tq2, x, u)
    check_sample(tq2, x, u, top_k=[vocab // 2 + 1 + r for r in range(rows)] if vocab > 200 else None)
    check_sample(tq2, x, u, top_p=[0.02 + r / 70 for r in range(rows)])


def test_sample_ends_of_the_range(tq2):
    rng = np.random.default_rng(9)
    x = logits_of(rng, 1, 5000, "f32")
    for u in (0.0, 2.0 ** -149, 1 - 2.0 ** -24, 1.0, 7.0, INF, NAN, -1.0, -INF):
        check_sample(tq2, x, [u])
        check_sample(tq2, x, [u], top_k=[40], top_p=[0.9])
    top = int(x[0].argmax())
    for f in (dict(temperature=[0.0]), dict(temperature=[-1.0]), dict(temperature=[NAN]), dict(temperature=[1e-38]),
              dict(top_k=[1]), dict(top_p=[0.0]), dict(top_p=[-2.0]), dict(top_p=[1e-9]), dict(min_p=[1.0]), dict(min_p=[9.0])):
        t, p = tq2.sample(x, torch.tensor([0.999], device="cuda"), **{
            k: torch.tensor(v, device="cuda", dtype=torch.int32 if k == "top_k" else torch.float32) for k, v in f.items()})
        assert int(t) == top and float(p) == 1.0, f
    for f in (dict(top_k=[0]), dict(top_k=[-3]), dict(top_k=[5000]), dict(top_k=[2 ** 31 - 1]), dict(top_p=[1.0]),
              dict(top_p=[INF]), dict(min_p=[0.0]), dict(min_p=[-INF])):
        check_sample(tq2, x, [0.8], **f)
    t, _ = tq2.sample(x, torch.tensor([0.5], device="cuda"), top_p=torch.tensor([NAN], device="cuda"),
                      min_p=torch.tensor([NAN], device="cuda"))
    assert int(t) == decode.sample(x[0].double().cpu().numpy(), 0.5)[0]
    t, p = tq2.sample(x, torch.tensor([0.5], device="cuda"), temperature=torch.tensor([INF], device="cuda"))
    assert abs(float(p) * 5000 - 1) < 1e-6  # every finite logit weighs the same


def test_sample_masked_rows(tq2):
    x = torch.full((8, 3000), -INF, device="cuda")
    x[1, 2999] = -1e30
    x[2, 5], x[2, 2000] = 1.0, 1.0
    x[3] = NAN
    x[4] = NAN
    x[4, 77] = 0.0
    x[5, 10], x[5, 11], x[5, 12] = INF, 3.0, INF
    x[6, 1:4] = torch.tensor([-3.4e38, 3.4e38, 0.0])
    x[7] = 0.0
    x[7, ::2] = -0.0
    u = [0.6] * 8
    for f in ({}, dict(top_k=[50] * 8), dict(top_p=[0.9] * 8), dict(min_p=[0.1] * 8)):
        check_sample(tq2, x, u, **f)
    t, p = tq2.sample(x, torch.tensor(u, device="cuda"))
    assert t.tolist()[:7] == [-1, 2999, 2000, -1, 77, 12, 2] and p.tolist()[0] == p.tolist()[3] == 0.0


def test_sample_many_equal_at_the_border(tq2):
    """Borders inside runs of equal logits, and logits so near each other that they share all coarse digits."""
    rng = np.random.default_rng(11)
    near = 5.0 + np.arange(20_000, dtype=np.float32) * np.float32(2.0 ** -21)  # steps of one ulp
    rows = np.stack([rng.permutation(near), rng.permutation(np.repeat(near[:20], 1000)),
                     np.where(np.arange(20_000) % 3 == 0, 4.0, 3.999).astype(np.float32)])
    x = torch.from_numpy(rows.astype(np.float32)).cuda()
    for u in (0.1, 0.5, 0.93):
        for f in ({}, dict(top_k=[777] * 3), dict(top_k=[9999] * 3, top_p=[0.37] * 3), dict(top_p=[0.5] * 3)):
            check_sample(tq2, x, [u] * 3, **f)


def test_sample_without_prob_given_outputs_stream_and_replay(tq2):
    rng = np.random.default_rng(12)
    x = logits_of(rng, 19, 12_345, "f16")
    u = torch.rand(19, device="cuda")
    k = torch.full((19,), 30, dtype=torch.int32, device="cuda")
    want, wp = tq2.sample(x, u, top_k=k)
    out, prob = torch.full((19,), -5, dtype=torch.int64, device="cuda"), torch.full((19,), NAN, device="cuda")
    tq2.tq2_sample(x, tq2.TQ2_F16, 12_345, u, tq2.tq2_sampling(top_k=k), out, None, 19, 12_345)
    assert torch.equal(out, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out.fill_(-5)
    side.wait_stream(torch.cuda.current_stream())
    got = tq2.sample(x, u, top_k=k, out=out, prob=prob, stream=side)
    side.synchronize()
    assert got[0] is out and torch.equal(out, want) and torch.equal(prob, wp)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tq2.sample(x, u, top_k=k, out=out, prob=prob)
    for seed in (13, 14):
        x.copy_(logits_of(np.random.default_rng(seed), 19, 12_345, "f16"))
        u.copy_(torch.rand(19, device="cuda"))
        k.fill_(seed)
        graph.replay()
        want, wp = tq2.sample(x, u, top_k=k)
        assert torch.equal(out, want) and torch.equal(prob, wp)


def test_sample_frequencies(tq2):
    """Many draws of one row: each token as often as its probability says (six standard deviations)."""
    n, vocab = 20_000, 50
    rng = np.random.default_rng(15)
    row = rng.standard_normal(vocab).astype(np.float32)
    x = torch.from_numpy(row).cuda()[None].expand(n, vocab).contiguous()
    t, _ = tq2.sample(x, torch.rand(n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)))
    p = np.exp(row.astype(np.float64) - row.max())
    p /= p.sum()
    count = np.bincount(t.cpu().numpy(), minlength=vocab)
    assert np.all(np.abs(count - n * p) <= 6 * np.sqrt(n * p * (1 - p)) + 1)


def test_sample_rows_past_32_bits(tq2):
    """Row offsets of more than 2^31 elements."""
    base = torch.empty(2 ** 31 + 4096, dtype=torch.float16, device="cuda")
    x = base.as_strided((2, 1000), (2 ** 31 + 8, 1))
    x.copy_(logits_of(np.random.default_rng(16), 2, 1000, "f16"))
    check_sample(tq2, x, [0.3, 0.7], top_k=[50, 0])
    e, w = tq2.moe_route(x, 5)
    we, _ = decode.route(x.double().cpu().numpy(), 5)
    assert np.array_equal(e.cpu().numpy(), we)

"""Mixtures of ternary experts on a GB300 against the 64-bit oracle."""

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


def soa(rng, rows, cols, high=3, spread=1.0):
    """A ternary weight in the device layout: codes below `high`, scales of either sign about cols^-0.5."""
    codes = rng.integers(0, high, (4, rows * cols // 4), dtype=np.uint8)
    d = (np.exp(rng.standard_normal(rows * cols // 128) * 0.3 * spread) * cols ** -0.5 * rng.choice([1, 1, 1, -1], rows * cols // 128))
    return np.concatenate([codes[0] | codes[1] << 2 | codes[2] << 4 | codes[3] << 6, d.astype(np.float16).view(np.uint8)])


class Layer:
    def __init__(self, tq2, experts, width, ffn, seed=0, high=3):
        rng = np.random.default_rng(seed)
        gu, dn = soa(rng, experts * 2 * ffn, width, high), soa(rng, experts * width, ffn, high)
        self.n, self.width, self.ffn = experts, width, ffn
        self.gu, self.dn = decode.matrices(gu, experts, 2 * ffn, width), decode.matrices(dn, experts, width, ffn)
        self.dev = tq2.Experts(torch.from_numpy(gu).cuda(), torch.from_numpy(dn).cuda(), experts=experts, width=width, ffn=ffn)


def routed(rng, tokens, experts, top_k, dropped=0.1):
    expert = np.stack([rng.permutation(experts)[:top_k] for _ in range(tokens)]).astype(np.int32).reshape(tokens, top_k)
    expert[rng.random(expert.shape) < dropped] = -1
    return expert, rng.uniform(-0.2, 1.0, (tokens, top_k)).astype(np.float32)


# What a result may be off by, relative to the oracle's `hidden`, `sums` and the result (see oracle.decode.experts):
#  hidden: 16-bit activations go to the second product in binary16 (half a step: 2^-11), f32 ones as two such terms (2^-22);
#          the activation itself is evaluated in f32 (2^-20 with the fast exponential and quotient).
#  sums:   products are exact, sums of them f32: at most 128 of a block, one of each block (up to 8 here), the pairs of a token
#          (up to 8) and the residual: 2^-24 each, half of them rounded the same way at worst: 96 * 2^-24.  An activation's
#          first term is exact in binary16 (f16), or within 2^-24 of the row's largest (bf16: what is below it by 2^21 or more
#          loses bits; f32: two terms, 2^-22 of itself, or 2^-31 of the row's largest).
#  result: one rounding to its type.
HIDDEN = {"f32": 2.0 ** -22 + 2.0 ** -20, "f16": 2.0 ** -11 + 2.0 ** -20, "bf16": 2.0 ** -11 + 2.0 ** -20}
SUMS = 96 * 2.0 ** -24 + 2.0 ** -22


def check(layer, out, dtype, x, expert, weight, residual=None):
    """The output against the oracle's, for the inputs as the device holds them."""
    ref, hidden, sums = decode.experts(layer.gu, layer.dn, x.double().cpu().numpy(), expert, weight,
                                       None if residual is None else residual.double().cpu().numpy())
    got = out.double().cpu().numpy()
    half = torch.finfo(DTYPES[dtype]).eps / 2
    tol = HIDDEN[dtype] * hidden + SUMS * sums + half * np.abs(ref) + 2.0 ** -25
    assert np.all(np.isfinite(got))
    worst = np.max(np.abs(got - ref) / tol)
    assert worst <= 1.0, worst
    # roundings are as often up as down: in the mean the result is much nearer than at worst
    typical = {"f32": 2.0 ** -20, "f16": 2.0 ** -11, "bf16": 2.0 ** -8.5}[dtype]
    # (binary16 results below 2^-14 are multiples of 2^-24: half a step, 2^-25, each)
    assert np.linalg.norm(got - ref) <= typical * np.sqrt(np.sum(ref ** 2) + np.sum(hidden ** 2) / layer.ffn) + 2.0 ** -25 * ref.size ** 0.5


def run(tq2, layer, dtype, tokens, top_k, seed=0, residual=True, dropped=0.1, sharp=1.0, workspace=True):
    rng = np.random.default_rng(seed + tokens)
    x = torch.from_numpy(rng.standard_normal((tokens, layer.width)) * sharp).to(DTYPES[dtype]).cuda()
    r = torch.from_numpy(rng.standard_normal((tokens, layer.width))).to(DTYPES[dtype]).cuda() if residual else None
    expert, weight = routed(rng, tokens, layer.n, top_k, dropped)
    ws = tq2.moe_swiglu_workspace(layer.dev, tokens, top_k, DTYPES[dtype]) if workspace else None
    if ws is not None:
        ws.fill_(0xFF)  # NaN in every type
    out = torch.full((tokens, layer.width), NAN, dtype=DTYPES[dtype], device="cuda")
    got = tq2.moe_swiglu(layer.dev, x, torch.from_numpy(expert).cuda(), torch.from_numpy(weight).cuda(), residual=r, out=out,
                         workspace=ws)
    assert got is out and tq2.tq2_device_status() == tq2.TQ2_OK
    check(layer, out, dtype, x, expert, weight, r)
    return x, r, expert, weight, out


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("experts,width,ffn", [(1, 128, 128), (4, 256, 384), (7, 640, 128), (3, 128, 640), (16, 1024, 256)])
@pytest.mark.parametrize("tokens", [1, 2, 3, 8, 17, 40])
def test_experts(tq2, dtype, experts, width, ffn, tokens):
    run(tq2, Layer(tq2, experts, width, ffn, seed=experts), dtype, tokens, min(experts, 3), residual=tokens % 2 == 0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens", [15, 16, 31, 32, 33, 63, 64, 65, 127, 128, 129, 130, 257, 300])
def test_tokens_of_one_expert(tq2, dtype, tokens):
    """All tokens at one expert: rows around every tile's size."""
    run(tq2, Layer(tq2, 1, 256, 256, seed=2), dtype, tokens, 1, dropped=0.0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("experts,width,ffn,tokens", [(40, 512, 768, 60), (64, 128, 1408, 130), (24, 2304, 640, 9),
                                                      (3, 1664, 4096, 400)])
def test_more_work_than_one_turn_of_the_gpu(tq2, dtype, experts, width, ffn, tokens):
    """Several items a CTA, odd numbers of blocks, every ring wrapping."""
    run(tq2, Layer(tq2, experts, width, ffn, seed=experts), dtype, tokens, 3)


@pytest.mark.parametrize("dtype", DTYPES)
def test_many_tokens_uneven(tq2, dtype):
    """Experts with hundreds of tokens beside experts with none or one."""
    layer, rng = Layer(tq2, 9, 384, 256, seed=3), np.random.default_rng(4)
    tokens, top_k = 700, 2
    x = torch.from_numpy(rng.standard_normal((tokens, 384))).to(DTYPES[dtype]).cuda()
    expert = np.where(rng.random((tokens, 2)) < 0.8, [[2, 5]], rng.choice([0, 7, -1], (tokens, 2))).astype(np.int32)
    expert[13, 1] = 8
    weight = rng.uniform(0, 1, (tokens, 2)).astype(np.float32)
    out = tq2.moe_swiglu(layer.dev, x, torch.from_numpy(expert).cuda(), torch.from_numpy(weight).cuda())
    check(layer, out, dtype, x, expert, weight)
    assert tq2.tq2_device_status() == tq2.TQ2_OK


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("sharp", [1e-4, 1e-2, 30.0])
def test_small_and_large_activations(tq2, dtype, sharp):
    run(tq2, Layer(tq2, 4, 256, 256, seed=5), dtype, 20, 2, residual=False, sharp=sharp)


def test_wide_range_within_a_row(tq2):
    """f32 and bf16 values far outside binary16's range, and rows whose values span it."""
    layer, rng = Layer(tq2, 2, 256, 128, seed=6), np.random.default_rng(7)
    for dtype, scale in (("f32", 1e5), ("bf16", 1e6), ("f32", 1e-7), ("bf16", 1e-6)):
        x = rng.standard_normal((6, 256)) * scale
        x[3:] *= 2.0 ** rng.integers(-12, 1, (3, 256))
        xt = torch.from_numpy(x).to(DTYPES[dtype]).cuda()
        expert, weight = routed(rng, 6, 2, 2, 0.0)
        out = tq2.moe_swiglu(layer.dev, xt, torch.from_numpy(expert).cuda(), torch.from_numpy(weight).cuda())
        ref, hidden, sums = decode.experts(layer.gu, layer.dn, xt.double().cpu().numpy(), expert, weight)
        got = out.double().cpu().numpy()
        half = torch.finfo(DTYPES[dtype]).eps / 2
        assert np.all(np.abs(got - ref) <= HIDDEN[dtype] * hidden + SUMS * sums + half * np.abs(ref) + 1e-30), (dtype, scale)


def test_code_three_and_zero_scales(tq2):
    layer = Layer(tq2, 3, 256, 128, seed=8, high=4)  # code 3 decodes as +2
    run(tq2, layer, "f32", 9, 2)
    run(tq2, layer, "bf16", 9, 2)
    rng = np.random.default_rng(9)
    gu, dn = soa(rng, 2 * 128, 128), soa(rng, 128, 128)
    gu[-2 * 2 * 128:] = 0  # every scale 0: nothing but the residual
    dev = tq2.Experts(torch.from_numpy(gu).cuda(), torch.from_numpy(dn).cuda(), experts=1, width=128, ffn=128)
    x, r = (torch.randn(5, 128, device="cuda") for _ in range(2))
    one = torch.zeros((5, 1), dtype=torch.int32, device="cuda")
    assert torch.equal(tq2.moe_swiglu(dev, x, one, torch.ones((5, 1), device="cuda"), residual=r), r)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens", [1, 6, 200])
def test_no_expert_at_all(tq2, dtype, tokens):
    layer = Layer(tq2, 2, 128, 128)
    x = torch.randn(tokens, 128, device="cuda").to(DTYPES[dtype])
    none = torch.full((tokens, 2), -1, dtype=torch.int32, device="cuda")
    w = torch.full((tokens, 2), NAN, device="cuda")  # (weights of no expert are not looked at)
    assert torch.equal(tq2.moe_swiglu(layer.dev, x, none, w), torch.zeros_like(x))
    r = torch.randn(tokens, 128, device="cuda").to(DTYPES[dtype])
    assert torch.equal(tq2.moe_swiglu(layer.dev, x, none, w, residual=r), r)
    assert tq2.tq2_device_status() == tq2.TQ2_OK
    assert tq2.moe_swiglu(layer.dev, x[:0], none[:0], w[:0]).shape == (0, 128)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens", [5, 150])
def test_bad_experts_count_as_none(tq2, dtype, tokens):
    layer, rng = Layer(tq2, 4, 128, 256, seed=10), np.random.default_rng(11)
    x = torch.from_numpy(rng.standard_normal((tokens, 128))).to(DTYPES[dtype]).cuda()
    expert, weight = routed(rng, tokens, 4, 3)
    expert[2] = [4, -2, 1]
    expert[4] = [2 ** 31 - 1, -2 ** 31, 1 << 20]
    out = tq2.moe_swiglu(layer.dev, x, torch.from_numpy(expert).cuda(), torch.from_numpy(weight).cuda())
    assert tq2.tq2_device_status() == tq2.TQ2_ERR_BAD_BATCH
    assert tq2.tq2_device_status() == tq2.TQ2_OK
    check(layer, out, dtype, x, expert, weight)


@pytest.mark.parametrize("dtype", DTYPES)
def test_same_expert_twice(tq2, dtype):
    layer, rng = Layer(tq2, 3, 256, 128, seed=12), np.random.default_rng(13)
    for tokens in (4, 90):
        x = torch.from_numpy(rng.standard_normal((tokens, 256))).to(DTYPES[dtype]).cuda()
        expert = np.full((tokens, 4), 1, dtype=np.int32)
        expert[::2, 2] = 0
        weight = rng.uniform(0, 1, expert.shape).astype(np.float32)
        out = tq2.moe_swiglu(layer.dev, x, torch.from_numpy(expert).cuda(), torch.from_numpy(weight).cuda())
        check(layer, out, dtype, x, expert, weight)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens", [3, 140])
def test_in_place_residual_no_workspace_and_same_bits(tq2, dtype, tokens):
    layer = Layer(tq2, 5, 256, 384, seed=14)
    x, r, expert, weight, out = run(tq2, layer, dtype, tokens, 3, seed=15)
    e, w = torch.from_numpy(expert).cuda(), torch.from_numpy(weight).cuda()
    for _ in range(3):
        place = r.clone()
        assert tq2.moe_swiglu(layer.dev, x, e, w, residual=place, out=place) is place
        assert torch.equal(place, out)
    own = tq2.moe_swiglu(layer.dev, x, e, w, residual=x)
    place = x.clone()
    tq2.moe_swiglu(layer.dev, place, e, w, residual=place, out=place)
    assert torch.equal(place, own)


@pytest.mark.parametrize("dtype,tokens", [("f16", 3), ("f16", 32), ("bf16", 3), ("bf16", 32), ("f32", 3), ("f32", 150)])
def test_a_token_alone_gets_the_same_result(tq2, dtype, tokens):
    """A token's result does not depend on the tokens beside it: the order and kind of its sums are its own (of 16-bit
    activations, as long as experts have no more than 16 rows in the mean, or have more)."""
    layer = Layer(tq2, 4, 256, 256, seed=16)
    x, r, expert, weight, out = run(tq2, layer, dtype, tokens, 2, seed=17)
    e, w = torch.from_numpy(expert).cuda(), torch.from_numpy(weight).cuda()
    for t in (0, 1, tokens - 1):
        alone = tq2.moe_swiglu(layer.dev, x[t:t + 1], e[t:t + 1], w[t:t + 1], residual=r[t:t + 1])
        assert torch.equal(alone[0], out[t])
    if dtype != "f32":
        several = tq2.moe_swiglu(layer.dev, x.repeat(60, 1), e.repeat(60, 1), w.repeat(60, 1), residual=r.repeat(60, 1))
        assert torch.equal(several, several[:tokens].repeat(60, 1))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens", [6, 200])
def test_nan_and_infinity_stay_in_their_rows(tq2, dtype, tokens):
    layer = Layer(tq2, 4, 256, 256, seed=18)
    x, r, expert, weight, out = run(tq2, layer, dtype, tokens, 2, seed=19, dropped=0.0)
    y = x.clone()
    y[1, 7], y[3, 200] = NAN, INF
    e, w = torch.from_numpy(expert).cuda(), torch.from_numpy(weight).cuda()
    got = tq2.moe_swiglu(layer.dev, y, e, w, residual=r)
    rest = [t for t in range(tokens) if t not in (1, 3)]
    assert torch.equal(got[rest], out[rest])
    assert torch.isnan(got[1]).all()
    assert not torch.isfinite(got[3]).any()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tokens,top_k", [(1, 1), (5, 2), (70, 3), (300, 2)])
def test_guard_bands(tq2, dtype, tokens, top_k):
    layer, rng = Layer(tq2, 5, 256, 128, seed=20), np.random.default_rng(21)
    x = torch.from_numpy(rng.standard_normal((tokens, 256))).to(DTYPES[dtype]).cuda()
    expert, weight = routed(rng, tokens, 5, top_k)
    nbytes = tq2.tq2_moe_swiglu_workspace_bytes(layer.dev.packed, {"f32": 0, "f16": 1, "bf16": 2}[dtype], tokens, top_k)
    ws = torch.full((nbytes + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    buf = torch.full((tokens * 256 + 256,), 7.0, dtype=DTYPES[dtype], device="cuda")
    out = buf[128:-128].view(tokens, 256)
    tq2.moe_swiglu(layer.dev, x, torch.from_numpy(expert).cuda(), torch.from_numpy(weight).cuda(), out=out,
                   workspace=ws[256:-256])
    check(layer, out, dtype, x, expert, weight)
    assert bool((buf[:128] == 7).all()) and bool((buf[-128:] == 7).all())
    assert bool((ws[:256] == 0xA5).all()) and bool((ws[-256:] == 0xA5).all())


@pytest.mark.parametrize("dtype", DTYPES)
def test_stream_and_replay(tq2, dtype):
    """A captured call whose routing changes between replays, from none to all tokens at one expert."""
    layer, rng = Layer(tq2, 6, 256, 128, seed=22), np.random.default_rng(23)
    tokens, top_k = 33, 2
    x = torch.from_numpy(rng.standard_normal((tokens, 256))).to(DTYPES[dtype]).cuda()
    e = torch.full((tokens, top_k), -1, dtype=torch.int32, device="cuda")
    w = torch.zeros((tokens, top_k), device="cuda")
    out = torch.empty_like(x)
    ws = tq2.moe_swiglu_workspace(layer.dev, tokens, top_k, x.dtype)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    tq2.moe_swiglu(layer.dev, x, e, w, out=out, workspace=ws, stream=side)
    side.synchronize()
    assert not out.any()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tq2.moe_swiglu(layer.dev, x, e, w, out=out, workspace=ws)
    for expert in (np.full((tokens, top_k), 3, np.int32), routed(rng, tokens, 6, top_k)[0], np.full((tokens, top_k), -1, np.int32),
                   np.tile(np.array([[0, 5]], np.int32), (tokens, 1))):
        weight = rng.uniform(0, 1, expert.shape).astype(np.float32)
        e.copy_(torch.from_numpy(expert))
        w.copy_(torch.from_numpy(weight))
        x.copy_(torch.from_numpy(rng.standard_normal((tokens, 256))))
        graph.replay()
        check(layer, out, dtype, x, expert, weight)
    assert tq2.tq2_device_status() == tq2.TQ2_OK


@pytest.mark.parametrize("tokens", [5, 600])
def test_captured_without_a_workspace_and_beside_another_graph(tq2, tokens):
    """A temporary of the graph's own in one graph, a workspace that both an eager call and another graph use in the other."""
    layer, rng = Layer(tq2, 4, 256, 128, seed=36), np.random.default_rng(37)
    x = torch.from_numpy(rng.standard_normal((tokens, 256))).to(torch.bfloat16).cuda()
    expert, weight = (torch.from_numpy(a).cuda() for a in routed(rng, tokens, 4, 2))
    want, outs, graphs = tq2.moe_swiglu(layer.dev, x, expert, weight), [], []
    ws = tq2.moe_swiglu_workspace(layer.dev, tokens, 2, x.dtype)
    for workspace in (None, ws):
        outs.append(torch.empty_like(x))
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            tq2.moe_swiglu(layer.dev, x, expert, weight, out=outs[-1], workspace=workspace)
    for _ in range(3):
        for out in outs:
            out.fill_(NAN)
        graphs[0].replay()
        graphs[1].replay()
        eager = tq2.moe_swiglu(layer.dev, x, expert, weight, workspace=ws)
        graphs[0].replay()
        assert torch.equal(outs[0], want) and torch.equal(outs[1], want) and torch.equal(eager, want)


def test_larger_workspace_serves_fewer_tokens(tq2):
    layer = Layer(tq2, 4, 256, 256, seed=24)
    ws = tq2.moe_swiglu_workspace(layer.dev, 300, 2, torch.bfloat16)
    rng = np.random.default_rng(25)
    for tokens in (300, 1, 40):
        x = torch.from_numpy(rng.standard_normal((tokens, 256))).to(torch.bfloat16).cuda()
        expert, weight = routed(rng, tokens, 4, 2)
        out = tq2.moe_swiglu(layer.dev, x, torch.from_numpy(expert).cuda(), torch.from_numpy(weight).cuda(), workspace=ws)
        check(layer, out, "bf16", x, expert, weight)


class Drawn:
    """A layer of random bytes drawn on the device; some experts' matrices for the oracle."""

    def __init__(self, tq2, experts, width, ffn, held):
        g = torch.Generator(device="cuda").manual_seed(experts)
        self.n, self.width, self.ffn, self.gu, self.dn = experts, width, ffn, {}, {}
        dev = []
        for rows, cols, to in ((2 * ffn, width, self.gu), (width, ffn, self.dn)):
            codes, blocks = rows * cols // 4, rows * cols // 128
            w = torch.empty(experts * (codes + 2 * blocks), dtype=torch.uint8, device="cuda")
            w[:experts * codes].random_(0, 256, generator=g)
            d = w[experts * codes:].view(torch.float16)
            d.uniform_(0.3 * cols ** -0.5, 1.2 * cols ** -0.5, generator=g)
            for e in held:
                one = torch.cat([w[e * codes:(e + 1) * codes], d[e * blocks:(e + 1) * blocks].view(torch.uint8)])
                to[e] = decode.matrices(one.cpu().numpy(), 1, rows, cols)[0]
            dev.append(w)
        self.dev = tq2.Experts(*dev, experts=experts, width=width, ffn=ffn)

    def some(self, expert):
        """The experts that `expert` names, and `expert` counting among these."""
        held = sorted(self.gu)
        part = type("Part", (), dict(gu=np.stack([self.gu[e] for e in held]), dn=np.stack([self.dn[e] for e in held]), ffn=self.ffn))
        return part, np.searchsorted(held, expert)


@pytest.mark.parametrize("dtype", DTYPES)
def test_weights_past_32_bits(tq2, dtype):
    """Codes of more than 2^32 bytes: the first and the last experts."""
    layer, rng = Drawn(tq2, 1024, 2048, 4096, (0, 511, 1000, 1023)), np.random.default_rng(28)
    x = torch.from_numpy(rng.standard_normal((6, 2048))).to(DTYPES[dtype]).cuda()
    expert = np.array([[0, 1023], [1023, 511], [1000, 1023], [511, 0], [1023, 1000], [1000, 0]], np.int32)
    weight = rng.uniform(0, 1, expert.shape).astype(np.float32)
    out = tq2.moe_swiglu(layer.dev, x, torch.from_numpy(expert).cuda(), torch.from_numpy(weight).cuda())
    part, among = layer.some(expert)
    check(part, out, dtype, x, among, weight)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_activations_past_32_bits(tq2, dtype):
    """Pairs times features of more than 2^31: the first and the last tokens."""
    tokens, width = 300_000, 4096
    layer = Layer(tq2, 2, width, 128, seed=29)
    g = torch.Generator(device="cuda").manual_seed(30)
    x = torch.empty((tokens, width), dtype=DTYPES[dtype], device="cuda").normal_(generator=g)
    expert = torch.randint(0, 2, (tokens, 2), dtype=torch.int32, device="cuda", generator=g)
    weight = torch.rand((tokens, 2), device="cuda", generator=g)
    out = tq2.moe_swiglu(layer.dev, x, expert, weight)
    at = [0, 1, 131_072, tokens // 2, tokens - 2, tokens - 1]
    check(layer, out[at], dtype, x[at], expert[at].cpu().numpy(), weight[at].cpu().numpy())


@pytest.mark.parametrize("dtype", ["f32", "f16"])
def test_most_pairs_of_most_experts(tq2, dtype):
    tokens, top_k, n = 1 << 17, 32, 1024
    layer, rng = Layer(tq2, n, 128, 128, seed=31), np.random.default_rng(32)
    x = torch.from_numpy(rng.standard_normal((tokens, 128)).astype(np.float32)).to(DTYPES[dtype]).cuda()
    expert = ((rng.integers(0, n, (tokens, 1)) + rng.integers(0, n // 2, (tokens, 1)) * 2 * np.arange(top_k) + np.arange(top_k)) % n).astype(np.int32)
    weight = rng.uniform(0, 1 / 16, (tokens, top_k)).astype(np.float32)
    out = tq2.moe_swiglu(layer.dev, x, torch.from_numpy(expert).cuda(), torch.from_numpy(weight).cuda())
    at = rng.integers(0, tokens, 60).tolist() + [0, tokens - 1]
    check(layer, out[at], dtype, x[at], expert[at], weight[at])
    assert bool(torch.isfinite(out).all()) and tq2.tq2_device_status() == tq2.TQ2_OK


def test_calls_on_two_streams_at_once(tq2):
    layers = [Layer(tq2, 8, 512, 256, seed=33), Layer(tq2, 4, 256, 640, seed=34)]
    rng, streams = np.random.default_rng(35), [torch.cuda.Stream(), torch.cuda.Stream()]
    calls = []
    for layer, dtype, tokens in ((layers[0], "bf16", 30), (layers[1], "f32", 200)):
        x = torch.from_numpy(rng.standard_normal((tokens, layer.width))).to(DTYPES[dtype]).cuda()
        expert, weight = (torch.from_numpy(a).cuda() for a in routed(rng, tokens, layer.n, 2))
        logits, u = torch.from_numpy(rng.standard_normal((tokens, 20_000))).cuda().float(), torch.rand(tokens, device="cuda")
        want = tq2.moe_swiglu(layer.dev, x, expert, weight), *tq2.moe_route(x, 8), *tq2.sample(logits, u)
        calls.append((layer, x, expert, weight, logits, u, want, []))
    torch.cuda.synchronize()
    for _ in range(20):
        for s, (layer, x, expert, weight, logits, u, _, got) in zip(streams, calls):
            got.append((tq2.moe_swiglu(layer.dev, x, expert, weight, stream=s), *tq2.moe_route(x, 8, stream=s),
                        *tq2.sample(logits, u, stream=s)))
    torch.cuda.synchronize()
    for *_, want, got in calls:
        for one in got:
            assert all(torch.equal(a, b) for a, b in zip(one, want))


def test_router_experts_sampling_together(tq2):
    """As they are used: logits of a router, its experts, and a token drawn from what comes out."""
    layer, rng = Layer(tq2, 8, 256, 128, seed=26), np.random.default_rng(27)
    for dtype in ("f32", "bf16"):
        x = torch.from_numpy(rng.standard_normal((21, 256))).to(DTYPES[dtype]).cuda()
        logits = (x.float() @ torch.from_numpy(rng.standard_normal((256, 8)) / 16).float().cuda()).to(DTYPES[dtype])
        expert, weight = tq2.moe_route(logits, 2, sigmoid=dtype == "bf16")
        out = tq2.moe_swiglu(layer.dev, x, expert, weight, residual=x)
        we, ww = decode.route(logits.double().cpu().numpy(), 2, dtype == "bf16")
        assert np.array_equal(we, expert.cpu().numpy())
        check(layer, out, dtype, x, we, ww.astype(np.float32), x)
        u = rng.random(21).astype(np.float32)
        t, p = tq2.sample(out, torch.from_numpy(u).cuda(), top_k=torch.full((21,), 9, dtype=torch.int32, device="cuda"))
        for r in range(21):
            want, wp, margin = decode.sample(out[r].double().cpu().numpy(), float(u[r]), top_k=9)
            assert margin < 4e-9 or (int(t[r]) == want and abs(float(p[r]) - wp) <= wp * 2.0 ** -23)


@pytest.mark.parametrize("dtype", DTYPES)
def test_uploaded_weights(tq2, dtype):
    """Weights quantised and uploaded by the library's own functions."""
    e, k, f = 3, 256, 128
    gen = torch.Generator(device="cuda").manual_seed(3)

    def ternary(rows, cols):
        w = torch.randn((rows, cols), device="cuda", generator=gen) * cols ** -0.5
        aos = torch.empty(tq2.tq2_soa_bytes(rows, cols), dtype=torch.uint8, device="cuda")
        tq2.tq2_quantize_f32(w, aos, rows, cols)
        return tq2.upload_weight(aos.cpu(), rows, cols)

    gu, dn = ternary(e * 2 * f, k), ternary(e * k, f)
    x = torch.randn((4, k), device="cuda", generator=gen).to(DTYPES[dtype])
    layer = Layer(tq2, e, k, f)
    layer.gu, layer.dn = decode.matrices(gu.cpu().numpy(), e, 2 * f, k), decode.matrices(dn.cpu().numpy(), e, k, f)
    layer.dev = tq2.Experts(gu, dn, experts=e, width=k, ffn=f)
    expert, weight = routed(np.random.default_rng(1), 4, e, 2)
    out = tq2.moe_swiglu(layer.dev, x, torch.from_numpy(expert).cuda(), torch.from_numpy(weight).cuda())
    check(layer, out, dtype, x, expert, weight)
    with pytest.raises(ValueError):
        tq2.Experts(gu, dn, experts=2, width=k, ffn=f)
    with pytest.raises(ValueError):
        tq2.moe_swiglu(layer.dev, x[:, :128], torch.from_numpy(expert).cuda(), torch.from_numpy(weight).cuda())
    with pytest.raises(ValueError):
        tq2.moe_swiglu(layer.dev, x, torch.from_numpy(expert).cuda(), torch.from_numpy(weight[:3]).cuda())
    with pytest.raises(ValueError):
        tq2.moe_swiglu(layer.dev, x, torch.from_numpy(expert).cuda().long(), torch.from_numpy(weight).cuda())


@pytest.mark.parametrize("dtype,tokens", [("f32", 5), ("bf16", 5), ("f16", 300), ("f32", 300)])
def test_a_wait_that_runs_out_is_reported_and_the_context_goes_on(tq2, dtype, tokens):
    layer = Layer(tq2, 4, 512, 384, seed=30)
    x, r, expert, weight, good = run(tq2, layer, dtype, tokens, 2, seed=31)
    e, w = torch.from_numpy(expert).cuda(), torch.from_numpy(weight).cuda()
    limit = tq2.tq2_set_wait_timeout_ns(0)
    try:
        for _ in range(3):
            tq2.moe_swiglu(layer.dev, x, e, w, residual=r)
        assert tq2.tq2_device_status() in (tq2.TQ2_ERR_TIMEOUT, tq2.TQ2_OK)  # (a wait may find its phase in time)
    finally:
        tq2.tq2_set_wait_timeout_ns(limit)
    again = tq2.moe_swiglu(layer.dev, x, e, w, residual=r)
    assert tq2.tq2_device_status() == tq2.TQ2_OK
    assert torch.equal(again, good)


def test_a_decoder_with_experts_and_sampling(tq2):
    """Greedy decoding by graph replays follows the logits of one pass; sampling at temperature 0 is greedy decoding, and with
    a top-k draws from the k best."""
    import importlib.util
    import os
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "ternary_decoder.py")
    spec = importlib.util.spec_from_file_location("ternary_decoder", path)
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    model = ex.Decoder(layers=2, ffn=256, vocab=256, experts=6)
    rng = np.random.default_rng(0)
    prompts = [rng.integers(0, 256, n).tolist() for n in (70, 5, 33)]
    each = lambda v, t=torch.float32: torch.full((3,), v, dtype=t, device="cuda")  # noqa: E731
    greedy, _ = ex.generate(model, prompts, 6, chunk=32)
    cold, _ = ex.generate(model, prompts, 6, chunk=32, sampling=dict(temperature=each(0.0)))
    assert torch.equal(greedy, cold)
    drawn, _ = ex.generate(model, prompts, 6, chunk=32, sampling=dict(top_k=each(3, torch.int32)))
    for rows, most in ((greedy.tolist(), 1), (drawn.tolist(), 3)):
        for p, row in zip(prompts, rows):
            text = p + row
            seqs = ex.Sequences(1, len(text))
            logits = model.step(torch.tensor(text, device="cuda"), model.new_caches(seqs.pages), seqs.batch([len(text)]))
            for i, got in enumerate(row):
                at = logits[len(p) - 1 + i].double()
                # (near ties: activations in binary16, a cache in bf16, and experts chosen by logits that those move)
                assert at.topk(most).values[-1] - at[got] <= 0.25 * at.std(), (len(p), i)
    assert tq2.tq2_device_status() == tq2.TQ2_OK

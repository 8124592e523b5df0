"""GPU tests of routing, mixtures of experts and sampling where calls go wrong or nearly so: clusters of every size, calls of
several host threads, magnitudes at a bound, scales of a wide spread, waits that run out, the widest layers.  Where a test
needs a tolerance of its own, its derivation stands beside it."""

import numpy as np
import pytest

from oracle import decode
from test_moe_gpu import check

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def tq2():
    import dit_tq2_g128_gb300 as m
    return m


@pytest.mark.parametrize("rows,vocab", [(400, 10_000), (400, 30_001), (400, 60_002), (60, 120_003), (3, 16_385)])
def test_sampling_by_clusters_of_every_size(tq2, rows, vocab):
    """One to eight CTAs a row, more clusters than the GPU holds, calls that begin while others end."""
    rng = np.random.default_rng(vocab)
    x = torch.from_numpy(rng.standard_normal((rows, vocab)).astype(np.float32) * 2).cuda()
    u = torch.from_numpy(rng.random(rows).astype(np.float32)).cuda()
    k = torch.from_numpy(rng.integers(-20, 80, rows).astype(np.int32)).cuda()
    got = [tq2.sample(x, u, top_k=k) for _ in range(12)]
    for r in (0, rows // 2, rows - 1):
        want, wp, margin = decode.sample(x[r].double().cpu().numpy(), float(u[r]), top_k=int(k[r]))
        # (the weights' 2^-30 and the probability's rounding, as in test_sampling_gpu)
        assert margin < 4e-9 or (int(got[0][0][r]) == want and abs(float(got[0][1][r]) - wp) <= wp * 2.0 ** -23)
    for t, p in got[1:]:
        assert torch.equal(t, got[0][0]) and torch.equal(p, got[0][1])


# ---------------------------------------------------------------------------
# hidden values of a mixture: staged by a bound of them


class Scaled:
    """A layer of given codes (or of random ones below 3) and scales d(rng, rows, blocks); matrices for the oracle."""

    def __init__(self, tq2, experts, width, ffn, gate_up_scales, code=None, seed=0):
        rng = np.random.default_rng(seed)
        self.n, self.width, self.ffn = experts, width, ffn

        def soa(rows, cols, d, code):
            c = rng.integers(0, 3, (4, rows * cols // 4), dtype=np.uint8) if code is None else np.full((4, rows * cols // 4), code, np.uint8)
            q = c[0] | c[1] << 2 | c[2] << 4 | c[3] << 6
            return np.concatenate([q, d.astype(np.float16).reshape(-1).view(np.uint8)])

        gu = soa(experts * 2 * ffn, width, gate_up_scales(rng, experts * 2 * ffn, width // 128), code)
        dn = soa(experts * width, ffn, rng.uniform(0.5, 1.5, (experts * width, ffn // 128)) * ffn ** -0.5, None)
        self.gu, self.dn = decode.matrices(gu, experts, 2 * ffn, width), decode.matrices(dn, experts, width, ffn)
        self.dev = tq2.Experts(torch.from_numpy(gu).cuda(), torch.from_numpy(dn).cuda(), experts=experts, width=width, ffn=ffn)

    def run(self, tq2, x, dtype):
        """All tokens at expert 0, against the oracle."""
        xt = torch.from_numpy(x).to(DTYPES[dtype]).cuda()
        expert, weight = np.zeros((len(x), 1), np.int32), np.linspace(0.5, 1.0, len(x), dtype=np.float32)[:, None]
        out = tq2.moe_swiglu(self.dev, xt, torch.from_numpy(expert).cuda(), torch.from_numpy(weight).cuda())
        assert tq2.tq2_device_status() == tq2.TQ2_OK
        return xt, expert, weight, out


@pytest.mark.parametrize("dtype,tokens", [("f32", 3), ("f32", 150), ("f16", 3), ("f16", 40), ("bf16", 3), ("bf16", 150)])
@pytest.mark.parametrize("scale", [1.0, 1.5])
def test_hidden_values_at_their_bound(tq2, dtype, tokens, scale):
    """Code 3 is +2: gate and up reach twice the largest scale times the sum of |x|, in rows that one element outweighs and
    in rows of one sign.  Sums from just above a power of two to just below the next."""
    layer = Scaled(tq2, 1, 256, 128, lambda rng, r, b: np.full((r, b), scale), code=3)
    rng = np.random.default_rng(tokens)
    total = np.array([15.96, 8.01, 10.7, 1.0, 0.52, 3.97, 31.0, 0.1245])[np.arange(tokens) % 8] / scale
    x = np.zeros((tokens, 256))
    x[np.arange(tokens), rng.integers(0, 256, tokens)] = total
    x[1::3] = total[1::3, None] / 256
    check(layer, *(lambda xt, e, w, out: (out, dtype, xt, e, w))(*layer.run(tq2, x, dtype)))


def spike(rng, rows, blocks, by):
    """All scales equal but one."""
    d = np.full((rows, blocks), (128 * blocks) ** -0.5)
    d[rng.integers(rows), rng.integers(blocks)] *= by
    return d


SPREADS = {
    "one 100 times the rest": lambda rng, r, b: spike(rng, r, b, 100.0),
    "one 1000 times the rest": lambda rng, r, b: spike(rng, r, b, 1000.0),
    "log-normal": lambda rng, r, b: np.exp(1.3 * rng.standard_normal((r, b))) * (128 * b) ** -0.5,
    "a gate row 300 times the rest": lambda rng, r, b: np.where(np.arange(r)[:, None] == r // 3, 300.0, 1.0) * np.full((r, b), (128 * b) ** -0.5),
}


@pytest.mark.parametrize("dtype,tokens", [("f32", 4), ("f32", 40), ("f16", 40), ("bf16", 40), ("bf16", 4)])
@pytest.mark.parametrize("spread", SPREADS)
@pytest.mark.parametrize("width", [256, 1280, 4096])
def test_scales_of_a_wide_spread(tq2, dtype, tokens, spread, width):
    """Hidden values that a few of an expert's scales put far below their bound keep their bits (check's mean error; its bound
    for single elements counts the sums' roundings at their worst and is wider for wide layers)."""
    layer = Scaled(tq2, 1, width, 256, SPREADS[spread], seed=width)
    x = np.random.default_rng(tokens).standard_normal((tokens, width))
    xt, e, w, out = layer.run(tq2, x, dtype)
    check(layer, out, dtype, xt, e, w)


@pytest.mark.parametrize("dtype,tokens,by", [("f32", 4, 300.0), ("f32", 40, 300.0), ("f32", 40, 10_000.0), ("f16", 40, 300.0),
                                             ("bf16", 40, 300.0), ("bf16", 40, 10_000.0)])
@pytest.mark.parametrize("width", [256, 4096])
def test_a_large_gate_that_is_shut(tq2, dtype, tokens, by, width):
    """A gate row far above the others that every token holds below 0: it bounds the hidden values, and gives none of them."""
    layer = Scaled(tq2, 1, width, 256, lambda rng, r, b: np.where(np.arange(r)[:, None] == 100, by, 1.0) * np.full((r, b), (128 * b) ** -0.5),
                   seed=width)
    x = np.random.default_rng(tokens).standard_normal((tokens, width))
    x *= -np.sign(x @ layer.gu[0, 100])[:, None]
    xt, e, w, out = layer.run(tq2, x, dtype)
    check(layer, out, dtype, xt, e, w)


@pytest.mark.parametrize("tokens", [4, 60])
def test_the_activation_of_closed_gates_in_f32(tq2, tokens):
    """silu to a few units in the last place where it is an exponential's, gates of -14 to -2: gate_f = d_f x_0, up_f = x_1 = 1,
    and down the identity, all exact.

    Relative roundings: the exponential 2^-22 (2 units in the last place at most), 1 + e, the quotient and the terms' sum
    2^-24 each, the two terms 2^-23: 4.5 * 2^-23; and the staging's floor, 2^-50 of b^2 = (2 (|x_0| + 1))^2 max d."""
    ffn = 128
    d = (1.0 + np.arange(ffn) / 256).astype(np.float16)
    codes = np.ones((2 * ffn, 128), np.uint8)  # 1: zero
    codes[:ffn, 0], codes[ffn:, 1] = 2, 2

    def soa(codes, d):
        c = codes.reshape(len(codes), -1, 4)
        return torch.from_numpy(np.concatenate([(c[..., 0] | c[..., 1] << 2 | c[..., 2] << 4 | c[..., 3] << 6).reshape(-1),
                                                d.view(np.uint8)])).cuda()

    dev = tq2.Experts(soa(codes, np.concatenate([d, np.ones(ffn, np.float16)])),
                      soa(np.ones((128, 128), np.uint8) + np.eye(128, dtype=np.uint8), np.ones(128, np.float16)), experts=1, width=128, ffn=ffn)
    x = np.zeros((tokens, 128), np.float32)
    x[:, 0], x[:, 1] = -2 - np.round(np.linspace(0, 7, tokens) * 64) / 64, 1.0
    out = tq2.moe_swiglu(dev, torch.from_numpy(x).cuda(), torch.zeros((tokens, 1), dtype=torch.int32, device="cuda"),
                         torch.ones((tokens, 1), device="cuda"))
    want = decode.silu(x[:, :1].astype(np.float64) * d.astype(np.float64))
    floor = 2.0 ** -50 * (2 * (np.abs(x[:, :1]) + 1)) ** 2 * float(d.max())
    err = np.abs(out.double().cpu().numpy() - want)
    assert np.all(err <= 4.5 * 2.0 ** -23 * np.abs(want) + floor), np.max((err - floor) / np.abs(want)) * 2.0 ** 23


# ---------------------------------------------------------------------------
# layers larger than the L2


def large(tq2, tokens, dtype, seed, experts=8, width=8192, ffn=4096):
    """A layer of 142 + 71 MB, tokens of it with two experts each."""
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def weight(rows, cols):
        w = torch.randint(0, 256, (tq2.tq2_soa_bytes(rows, cols),), dtype=torch.uint8, device="cuda", generator=gen)
        w[rows * cols // 4:].view(torch.float16).uniform_(0.5 * cols ** -0.5, 1.5 * cols ** -0.5, generator=gen)
        return w

    layer = tq2.Experts(weight(experts * 2 * ffn, width), weight(experts * width, ffn), experts=experts, width=width, ffn=ffn)
    x = torch.randn((tokens, width), device="cuda", generator=gen).to(DTYPES[dtype])
    expert = ((torch.arange(tokens, device="cuda")[:, None] * 2 + torch.tensor([[0, 1]], device="cuda")) % experts).int().contiguous()
    return layer, x, expert, torch.ones((tokens, 2), device="cuda")


def in_64_bits(layer, x, expert, scale):
    """The layer's output by the formula, some rows of an expert's matrices at a time."""
    out = torch.zeros(x.shape, dtype=torch.float64, device="cuda")

    def product(soa, e, rows, cols, v):
        at, some, parts = layer.experts * rows * cols // 4, max(1, (1 << 28) // cols), []
        for r in range(e * rows, (e + 1) * rows, some):
            n = min(some, (e + 1) * rows - r)
            q = soa[r * cols // 4:(r + n) * cols // 4].view(n, cols // 4)
            c = torch.stack([q >> 2 * j & 3 for j in range(4)], -1).view(n, cols).double() - 1.0
            d = soa[at:].view(torch.float16).view(-1, cols // 128)[r:r + n].double()
            parts.append(v @ c.view(n, cols // 128, 128).mul_(d[:, :, None]).view(n, cols).T)
        return torch.cat(parts, 1)

    for e in range(layer.experts):
        t, j = (expert == e).nonzero(as_tuple=True)
        if t.numel():
            z = product(layer.gate_up, e, 2 * layer.ffn, layer.width, x[t].double())
            h = torch.nn.functional.silu(z[:, :layer.ffn]) * z[:, layer.ffn:]
            out.index_add_(0, t, product(layer.down, e, layer.width, layer.ffn, h) * scale[t, j].double()[:, None])
    return out


# What a result may be off by in the mean (norms; see test_moe_gpu.check).  f32 sums of up to 512 blocks are within it: each
# addition rounds by 2^-24 / 3^0.5 of a partial sum, (512 / 2)^0.5 of them are 5.5e-7 of gate and up, 7.8e-7 of h, as much
# again of down at its widest: 1.1e-6 together.
TYPICAL = {"f32": 2.0 ** -20, "f16": 2.0 ** -11, "bf16": 2.0 ** -8.5}


@pytest.mark.parametrize("dtype,tokens", [("f32", 3), ("f16", 3), ("bf16", 40), ("f32", 70)])
@pytest.mark.parametrize("experts,width,ffn", [(3, 4224, 4224), (2, 65_536, 128), (2, 128, 65_536), (2, 16_512, 8320), (1, 65_536, 65_536)])
def test_the_widest_layers(tq2, dtype, tokens, experts, width, ffn):
    layer, x, expert, scale = large(tq2, tokens, dtype, tokens, experts, width, ffn)
    got, ref = tq2.moe_swiglu(layer, x, expert, scale), in_64_bits(layer, x, expert, scale)
    assert tq2.tq2_device_status() == tq2.TQ2_OK
    assert float((got.double() - ref).norm()) <= TYPICAL[dtype] * 2 ** 0.5 * float(ref.norm())
    # and no column is wrong by itself
    far = ((got.double() - ref).abs() / ref.pow(2).mean(1, keepdim=True).sqrt()).max()
    assert float(far) <= 16 * TYPICAL[dtype]


@pytest.mark.parametrize("dtype,tokens", [("f32", 6), ("bf16", 6), ("f16", 150), ("f32", 300), ("bf16", 700)])
def test_codes_that_come_late_from_memory(tq2, dtype, tokens):
    """The same bits on every call, and the formula's values, where codes are awaited row by row from memory: a decoder that
    gave a stage back before it had read it took the next one's in its place.  (Mean errors as in test_moe_gpu.check.)"""
    layer, x, expert, scale = large(tq2, tokens, dtype, tokens)
    rest = torch.empty(300 << 20, dtype=torch.uint8, device="cuda")
    good = tq2.moe_swiglu(layer, x, expert, scale)
    ref = in_64_bits(layer, x, expert, scale)
    assert float((good.double() - ref).norm()) <= TYPICAL[dtype] * 2 ** 0.5 * float(ref.norm())
    for i in range(30):
        if i % 2:
            rest.fill_(i)  # (nothing of the layer is in the L2)
        assert torch.equal(tq2.moe_swiglu(layer, x, expert, scale), good), i
    assert tq2.tq2_device_status() == tq2.TQ2_OK


# ---------------------------------------------------------------------------
# waits


class Limit:
    """A limit on the device's waits, put back at the end."""

    def __init__(self, tq2, ns):
        self.tq2, self.ns = tq2, ns

    def __enter__(self):
        torch.cuda.synchronize()
        self.before = self.tq2.tq2_set_wait_timeout_ns(self.ns)

    def __exit__(self, *_):
        self.tq2.tq2_set_wait_timeout_ns(self.before)


@pytest.mark.parametrize("dtype,tokens", [("f32", 6), ("bf16", 6), ("f16", 150), ("f32", 300)])
def test_a_wait_of_the_experts_that_runs_out_is_reported(tq2, dtype, tokens):
    """Three items and more a CTA, of 64 blocks: the second group of sums waits for all of the first one's, some 10 us and more,
    which is longer than a poll sleeps."""
    layer, x, expert, scale = large(tq2, tokens, dtype, tokens)
    good = tq2.moe_swiglu(layer, x, expert, scale)
    assert tq2.tq2_device_status() == tq2.TQ2_OK
    for _ in range(5):
        with Limit(tq2, 0):
            tq2.moe_swiglu(layer, x, expert, scale)
            assert tq2.tq2_device_status() == tq2.TQ2_ERR_TIMEOUT
        assert tq2.tq2_device_status() == tq2.TQ2_OK
        assert torch.equal(tq2.moe_swiglu(layer, x, expert, scale), good)
    assert tq2.tq2_device_status() == tq2.TQ2_OK

"""Routing, mixtures of experts and sampling: the oracle's own checks, and what the entry points refuse (no GPU)."""

import numpy as np
import pytest

from oracle import decode

A = 1 << 20  # fake, aligned, non-overlapping "device" addresses
P = [A * (i + 1) * 64 for i in range(12)]


@pytest.fixture(scope="module")
def tq2():
    import __graft_entry__
    __graft_entry__.build()
    import dit_tq2_g128_gb300 as m
    return m


def test_oracle_order():
    v = np.array([1.0, np.nan, 3.0, -0.0, 0.0, 3.0, -np.inf])
    assert decode.order(v).tolist() == [2, 5, 0, 3, 4, 6, 1]


def test_oracle_sample_small():
    l = np.log(np.array([1.0, 4.0, 2.0, 1.0]))  # weights by order: 1:4, 2:2, 0:1, 3:1 of 8
    for u, want in ((0.0, 1), (0.49, 1), (0.51, 2), (0.74, 2), (0.76, 0), (0.874, 0), (0.876, 3), (0.9999, 3)):
        assert decode.sample(l, u)[0] == want
    assert decode.sample(l, 0.99, top_k=2)[0] == 2
    assert decode.sample(l, 0.99, top_p=0.4)[0] == 1
    assert decode.sample(l, 0.99, top_p=0.51)[0] == 2
    assert decode.sample(l, 0.99, min_p=0.3)[0] == 2
    assert decode.sample(l, 0.99, temperature=0.0)[0] == 1
    assert decode.sample(np.full(3, -np.inf), 0.5)[0] == -1
    token, p, _ = decode.sample(l, 0.3, top_k=2)
    assert token == 1 and abs(p - 4 / 6) < 1e-15


def test_oracle_experts_against_differences():
    """The oracle's layer is linear in the routing weights and follows the formula for one expert."""
    rng = np.random.default_rng(0)
    soa = lambda rows, cols: np.concatenate([  # noqa: E731
        rng.integers(0, 256, rows * cols // 4, dtype=np.uint8),
        rng.standard_normal(rows * cols // 128).astype(np.float16).view(np.uint8)])
    gu, dn = decode.matrices(soa(2 * 256, 128), 2, 256, 128), decode.matrices(soa(2 * 128, 128), 2, 128, 128)
    x = rng.standard_normal((3, 128))
    e = np.array([[0, 1], [1, -1], [-1, -1]])
    w = rng.standard_normal((3, 2))
    out, _, _ = decode.experts(gu, dn, x, e, w)
    g = gu[1] @ x[1]
    assert np.allclose(out[1], w[1, 0] * dn[1] @ (g[:128] / (1 + np.exp(-g[:128])) * g[128:]))
    assert not out[2].any()
    twice, _, _ = decode.experts(gu, dn, x, e, 2 * w)
    assert np.allclose(twice, 2 * out)


# ---------------------------------------------------------------------------
# refusals (before any device is looked up)


def route(tq2, logits=P[0], dtype=0, stride=64, experts=P[1], weights=P[2], tokens=4, n=64, k=4, scale=1.0):
    return tq2.lib.tq2_moe_route(logits, dtype, stride, experts, weights, tokens, n, k, 0, 1, scale, None)


@pytest.mark.parametrize("change", [
    dict(logits=None), dict(experts=None), dict(weights=None), dict(dtype=3), dict(dtype=-1), dict(tokens=-1),
    dict(tokens=(1 << 24) + 1), dict(n=0), dict(n=1025, stride=2000), dict(k=0), dict(k=33), dict(k=65), dict(stride=63),
    dict(stride=-64), dict(scale=float("nan")), dict(scale=float("inf")), dict(experts=P[0]), dict(weights=P[0] + 1000),
    dict(weights=P[1] + 60)])
def test_route_refusals(tq2, change):
    assert route(tq2, **change) == tq2.TQ2_ERR_INVALID_ARG


@pytest.mark.parametrize("change", [dict(logits=P[0] + 2), dict(logits=P[0] + 1, dtype=2), dict(experts=P[1] + 2),
                                    dict(weights=P[2] + 1)])
def test_route_misaligned(tq2, change):
    assert route(tq2, **change) == tq2.TQ2_ERR_MISALIGNED


def test_route_of_no_tokens(tq2):
    assert route(tq2, tokens=0, logits=None, experts=None, weights=None) == tq2.TQ2_OK
    assert route(tq2, tokens=0, k=65) == tq2.TQ2_ERR_INVALID_ARG


def moe(tq2, gate_up=P[0], down=P[1], experts=4, width=256, ffn=128, x=P[2], expert=P[3], weight=P[4], residual=None,
        out=P[5], dtype=0, tokens=3, k=2, ws=None, ws_bytes=0):
    w = tq2.tq2_experts(gate_up, down, experts, width, ffn)
    return tq2.lib.tq2_moe_swiglu(w, x, expert, weight, residual, out, dtype, tokens, k, ws, ws_bytes, None)


@pytest.mark.parametrize("change", [
    dict(gate_up=None), dict(down=None), dict(x=None), dict(expert=None), dict(weight=None), dict(out=None),
    dict(experts=0), dict(experts=1025), dict(dtype=3), dict(tokens=-1), dict(k=0), dict(k=33), dict(tokens=1 << 22),
    dict(width=65536 + 128), dict(ffn=65536 + 128), dict(experts=1024, width=65536, ffn=65536), dict(out=P[2]),
    dict(out=P[3]), dict(out=P[4]), dict(out=P[0]), dict(out=P[1] + 4096), dict(residual=P[5] + 16),
    dict(ws=P[6], ws_bytes=16), dict(ws=P[5], ws_bytes=1 << 30), dict(ws=P[0], ws_bytes=1 << 30),
    dict(ws=P[4], ws_bytes=1 << 30)])
def test_moe_refusals(tq2, change):
    assert moe(tq2, **change) == tq2.TQ2_ERR_INVALID_ARG


@pytest.mark.parametrize("change", [dict(width=0), dict(width=-128), dict(width=200), dict(ffn=64), dict(ffn=0)])
def test_moe_bad_k(tq2, change):
    assert moe(tq2, **change) == tq2.TQ2_ERR_BAD_K


@pytest.mark.parametrize("change", [dict(gate_up=P[0] + 8), dict(down=P[1] + 2), dict(x=P[2] + 4), dict(out=P[5] + 8),
                                    dict(residual=P[7] + 8), dict(expert=P[3] + 2), dict(weight=P[4] + 1),
                                    dict(ws=P[6] + 8, ws_bytes=1 << 30)])
def test_moe_misaligned(tq2, change):
    assert moe(tq2, **change) == tq2.TQ2_ERR_MISALIGNED


def test_moe_of_no_tokens(tq2):
    assert moe(tq2, tokens=0, x=None, out=None) == tq2.TQ2_OK
    assert moe(tq2, tokens=0, width=100) == tq2.TQ2_ERR_BAD_K


def test_moe_workspace_bytes(tq2):
    w = tq2.tq2_experts(None, None, 8, 256, 384)
    got = [tq2.tq2_moe_swiglu_workspace_bytes(w, 0, t, 2) for t in (0, 1, 2, 5, 17, 64, 65, 300, 5000, 1 << 20)]
    assert got[0] == 0 and all(a <= b for a, b in zip(got, got[1:])) and got[1] > 0
    for bad in (tq2.tq2_experts(None, None, 8, 100, 384), tq2.tq2_experts(None, None, 0, 256, 384)):
        assert tq2.tq2_moe_swiglu_workspace_bytes(bad, 0, 5, 2) == 0
    assert tq2.tq2_moe_swiglu_workspace_bytes(w, 7, 5, 2) == 0
    assert tq2.tq2_moe_swiglu_workspace_bytes(w, 0, 5, 33) == 0


def sample(tq2, logits=P[0], dtype=0, stride=1000, u=P[1], temperature=None, top_k=None, top_p=None, min_p=None,
           tokens=P[2], prob=P[3], rows=4, vocab=1000):
    return tq2.lib.tq2_sample(logits, dtype, stride, u, tq2.tq2_sampling(temperature, top_k, top_p, min_p), tokens, prob,
                              rows, vocab, None)


@pytest.mark.parametrize("change", [
    dict(logits=None), dict(u=None), dict(tokens=None), dict(dtype=3), dict(rows=-1), dict(rows=(1 << 24) + 1),
    dict(vocab=0), dict(vocab=(1 << 18) + 1, stride=1 << 20), dict(stride=999), dict(stride=0), dict(tokens=P[0]),
    dict(prob=P[0]), dict(tokens=P[1]), dict(prob=P[1] + 8), dict(prob=P[2] + 8), dict(tokens=P[4], temperature=P[4]),
    dict(prob=P[4], top_k=P[4]), dict(tokens=P[4], top_p=P[4] + 8), dict(prob=P[4], min_p=P[4])])
def test_sample_refusals(tq2, change):
    assert sample(tq2, **change) == tq2.TQ2_ERR_INVALID_ARG


@pytest.mark.parametrize("change", [dict(logits=P[0] + 2), dict(logits=P[0] + 1, dtype=1), dict(u=P[1] + 2),
                                    dict(tokens=P[2] + 4), dict(prob=P[3] + 2), dict(temperature=P[4] + 1),
                                    dict(top_k=P[4] + 2), dict(top_p=P[4] + 2), dict(min_p=P[4] + 2)])
def test_sample_misaligned(tq2, change):
    assert sample(tq2, **change) == tq2.TQ2_ERR_MISALIGNED


def test_sample_of_no_rows(tq2):
    assert sample(tq2, rows=0, logits=None, u=None, tokens=None) == tq2.TQ2_OK


def test_host_memory_is_refused_or_no_device(tq2):
    """Memory that is not the current device's (here: no device at all) never reaches a launch."""
    assert route(tq2) in (tq2.TQ2_ERR_INVALID_ARG, tq2.TQ2_ERR_CUDA, tq2.TQ2_ERR_UNSUPPORTED_DEVICE)
    assert moe(tq2) in (tq2.TQ2_ERR_INVALID_ARG, tq2.TQ2_ERR_CUDA, tq2.TQ2_ERR_UNSUPPORTED_DEVICE)
    assert sample(tq2) in (tq2.TQ2_ERR_INVALID_ARG, tq2.TQ2_ERR_CUDA, tq2.TQ2_ERR_UNSUPPORTED_DEVICE)


def test_tensor_checks(tq2):
    """The tensor functions refuse what they cannot pass on, before any call."""
    torch = pytest.importorskip("torch")
    t = torch.zeros(4, 128)
    with pytest.raises(ValueError):
        tq2.moe_route(t, 2)  # a CPU tensor
    with pytest.raises(ValueError):
        tq2.sample(t, torch.zeros(4))
    with pytest.raises(ValueError):
        tq2.Experts(torch.zeros(tq2.tq2_soa_bytes(256, 128), dtype=torch.uint8), torch.zeros(1, dtype=torch.uint8),
                    experts=1, width=128, ffn=128)
    with pytest.raises(tq2.TQ2Error):
        tq2.Experts(t, t, experts=1, width=100, ffn=128)

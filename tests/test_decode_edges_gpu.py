"""GPU tests of routing, mixtures of experts and sampling where calls go wrong or nearly so: clusters of every size, calls of
several host threads, magnitudes at a bound, scales of a wide spread, waits that run out, the widest layers.  Where a test
needs a tolerance of its own, its derivation stands beside it."""

import numpy as np
import pytest

from oracle import decode

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

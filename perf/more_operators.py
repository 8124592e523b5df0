"""What a decoder's step of ternary layers does after its attention, as calls to be timed: routing tokens to experts, the
ternary experts' products, and sampling the next token.

``run`` computes them in elementary torch operations, or, where ``own`` is true, through the package.  Sizes follow from
the case alone; values and the routing follow from the seed.
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
BYTES = {"f32": 4, "f16": 2, "bf16": 2}


# ---------------------------------------------------------------------------
# cases


def listed():
    return [
        # one token of one conversation: launch latency
        dict(name="route one token", op="route", tokens=1, experts=64, top_k=6, dtype="f32", sigmoid=False,
             normalize=True, scale=1.0),
        # a prompt's tokens, many small experts, gates that do not compete
        dict(name="route prompt", op="route", tokens=8191, experts=256, top_k=8, dtype="bf16", sigmoid=True,
             normalize=True, scale=2.5),
        # one token of one conversation: six experts' weights, latency
        dict(name="experts one token", op="experts", tokens=1, experts=64, top_k=6, width=2048, ffn=1408, dtype="bf16",
             residual=True, padded=0),
        # a few conversations at once, few large experts: all weights are read
        dict(name="experts few tokens", op="experts", tokens=7, experts=8, top_k=2, width=4096, ffn=6144, dtype="f16",
             residual=False, padded=0),
        # decoding step of a batch, many small experts: about all weights are read, each for a few tokens
        dict(name="experts decode batch", op="experts", tokens=64, experts=128, top_k=8, width=2048, ffn=768,
             dtype="bf16", residual=True, padded=0),
        # drafted tokens in f32 towards f32 layers, the batch padded to a captured graph's size
        dict(name="experts drafts", op="experts", tokens=80, experts=32, top_k=4, width=1024, ffn=512, dtype="f32",
             residual=True, padded=5),
        # a chunk of a prompt in f32
        dict(name="experts chunk", op="experts", tokens=513, experts=16, top_k=2, width=1280, ffn=2816, dtype="f32",
             residual=False, padded=0),
        # a long prompt: compute counts
        dict(name="experts prompt", op="experts", tokens=4096, experts=64, top_k=8, width=2048, ffn=1024, dtype="bf16",
             residual=True, padded=0),
        # one conversation's next token, all filters: latency
        dict(name="sample one", op="sample", rows=1, vocab=32_000, dtype="f32", temperature=True, top_k=50, top_p=True,
             min_p=False, flat=False),
        # decoding step of a batch whose requests ask for different filters
        dict(name="sample batch", op="sample", rows=64, vocab=128_000, dtype="f32", temperature=True, top_k=-1,
             top_p=True, min_p=True, flat=False),
        # a large batch, 16-bit logits with many ties, an odd vocabulary (rows of any alignment), top-k alone
        dict(name="sample ties", op="sample", rows=256, vocab=100_003, dtype="bf16", temperature=True, top_k=100,
             top_p=False, min_p=False, flat=False),
        # creative sampling over a flat distribution and a large vocabulary: nothing is cut but a nucleus
        dict(name="sample flat", op="sample", rows=16, vocab=200_000, dtype="f16", temperature=True, top_k=0,
             top_p=True, min_p=False, flat=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "experts", "experts", "experts", "sample", "sample"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if op == "route":
        experts = rng.choice([8, 64, 128, 256, rng.randint(1, 512)])
        return dict(op=op, tokens=_log(rng, 1, 16_384), experts=experts, top_k=rng.randint(1, min(experts, 12)),
                    dtype=dtype, sigmoid=rng.random() < 0.5, normalize=rng.random() < 0.7,
                    scale=rng.choice([1.0, 1.0, 2.5]))
    if op == "experts":
        width, ffn = 128 * _log(rng, 1, 32), 128 * _log(rng, 1, 32)
        experts = _log(rng, 1, max(1, min(128, 400_000_000 // (3 * width * ffn))))
        top_k = rng.randint(1, min(experts, 8))
        most = 400_000_000_000 // (6 * width * ffn * top_k) // (2 if dtype == "f32" else 1)
        tokens = _log(rng, 1, max(1, min(4096, most)))
        return dict(op=op, tokens=tokens, experts=experts, top_k=top_k, width=width, ffn=ffn, dtype=dtype,
                    residual=rng.random() < 0.5, padded=rng.choice([0, 0, tokens // 7]))
    rows = _log(rng, 1, 256)
    vocab = _log(rng, 100, min(200_000, 25_000_000 // rows))
    return dict(op=op, rows=rows, vocab=vocab, dtype=dtype, temperature=rng.random() < 0.8,
                top_k=rng.choice([0, -1, _log(rng, 1, 1000)]), top_p=rng.random() < 0.6, min_p=rng.random() < 0.3,
                flat=rng.random() < 0.3)


# ---------------------------------------------------------------------------
# what a user's program has in hand


def _weight(gen, rows, cols):
    """A ternary weight in the device layout: codes [rows, cols / 4] (four a byte), then a binary16 scale per 128."""
    part = torch.randint(0, 3, (4, rows, cols // 4), generator=gen, device="cuda", dtype=torch.uint8)
    codes = part[0] | part[1] << 2 | part[2] << 4 | part[3] << 6
    d = torch.rand((rows, cols // 128), generator=gen, device="cuda").add_(0.5).mul_(1.2 * cols ** -0.5).half()
    return torch.cat([codes.view(-1), d.view(torch.uint8).view(-1)])


def _logits(gen, rows, vocab, flat):
    """Next-token logits: a few likely tokens and a long tail, sharper in some rows than in others."""
    x = torch.randn((rows, vocab), generator=gen, device="cuda")
    if flat:
        return x
    rank = torch.rand((rows, vocab), generator=gen, device="cuda").mul_(vocab).add_(1.0).log_()
    sharp = torch.linspace(0.8, 1.8, rows, device="cuda")[:, None]
    return (x * 0.7 - rank * 1.3 + 12.0) * sharp


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    dtype = DTYPES[case["dtype"]]
    if case["op"] == "route":
        popular = torch.randn((1, case["experts"]), generator=gen, device="cuda")
        x = torch.randn((case["tokens"], case["experts"]), generator=gen, device="cuda")
        s["logits"] = (x * 1.5 + popular * 0.5).to(dtype)
    elif case["op"] == "experts":
        n, e, k, f = case["tokens"], case["experts"], case["width"], case["ffn"]
        s["gate_up"] = _weight(gen, e * 2 * f, k)
        s["down"] = _weight(gen, e * k, f)
        s["x"] = torch.randn((n, k), generator=gen, device="cuda").to(dtype)
        s["skip"] = torch.randn((n, k), generator=gen, device="cuda").to(dtype) if case["residual"] else None
        score = torch.randn((n, e), generator=gen, device="cuda") + 0.5 * torch.randn((1, e), generator=gen, device="cuda")
        best = score.topk(case["top_k"], dim=1)
        s["expert"], s["weight"] = best.indices.to(torch.int32), best.values.softmax(1)
        if case["padded"]:
            s["expert"][n - case["padded"]:] = -1
        s["out"] = torch.empty((n, k), dtype=dtype, device="cuda")
    else:
        n, v = case["rows"], case["vocab"]
        s["logits"] = _logits(gen, n, v, case["flat"]).to(dtype)
        s["u"] = torch.rand(n, generator=gen, device="cuda")
        some = torch.rand((4, n), generator=gen, device="cuda")
        s["t"] = 0.5 + some[0] if case["temperature"] else None
        # -1: requests with and without a limit in one batch
        k = torch.full((n,), case["top_k"], dtype=torch.int32, device="cuda")
        s["k"] = None if case["top_k"] == 0 else k if case["top_k"] > 0 else (some[1] * 80 - 20).to(torch.int32)
        s["p"] = 0.7 + 0.3 * some[2] if case["top_p"] else None
        s["m"] = 0.1 * some[3] ** 2 if case["min_p"] else None
    if own:  # the handle and the workspace that such a program makes once and keeps
        import dit_tq2_g128_gb300 as tq2
        s["tq2"] = tq2
        if case["op"] == "experts":
            s["layer"] = tq2.Experts(s["gate_up"], s["down"], experts=case["experts"], width=case["width"], ffn=case["ffn"])
            s["workspace"] = tq2.moe_swiglu_workspace(s["layer"], case["tokens"], case["top_k"], dtype)
    return s


# ---------------------------------------------------------------------------
# one pass


def _route(s):
    x = s["logits"].float()
    order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :s["top_k"]]
    if s["sigmoid"]:
        score = 1.0 / (1.0 + torch.exp(-x))
    else:
        z = torch.exp(x - x.amax(1, keepdim=True))
        score = z / z.sum(1, keepdim=True)
    w = score.gather(1, order)
    if s["normalize"]:
        w = w / w.sum(1, keepdim=True)
    return order.to(torch.int32), w * s["scale"]


def _matrices(soa, experts, rows, cols, which):
    """f32 matrices [len(which), rows, cols] of some experts (None: of all) of a ternary weight."""
    at = experts * rows * cols // 4
    codes = soa[:at].view(experts, rows, cols // 4)
    d = soa[at:].view(torch.float16).view(experts, rows, cols // 128, 1)
    if which is not None:
        codes, d = codes[which], d[which]
    shift = torch.tensor([0, 2, 4, 6], dtype=torch.uint8, device=soa.device)
    c = (codes.unsqueeze(-1) >> shift & 3).to(torch.float32).sub_(1.0)
    return c.view(-1, rows, cols // 128, 128).mul_(d.float()).view(-1, rows, cols)


def _experts(s):
    n, e, k, f, top = s["tokens"], s["experts"], s["width"], s["ffn"], s["top_k"]
    x, dtype = s["x"].float(), s["x"].dtype
    pairs = s["expert"].reshape(-1).long()
    token = torch.arange(n * top, device=x.device) // top
    if n * top <= e:  # fewer pairs than experts: a matrix for each pair
        which = pairs.clamp(min=0)
        xg = x[token][:, :, None]
        gu = torch.bmm(_matrices(s["gate_up"], e, 2 * f, k, which), xg)[:, :, 0]
        h = gu[:, :f] / (1.0 + torch.exp(-gu[:, :f])) * gu[:, f:]
        y = torch.bmm(_matrices(s["down"], e, k, f, which), h[:, :, None])[:, :, 0]
    else:  # the pairs sorted by expert, padded to the most that one has
        order = torch.argsort(pairs, stable=True)
        mine = pairs[order]
        count = torch.zeros(e + 1, dtype=torch.int64, device=x.device).index_add_(0, mine + 1, torch.ones_like(mine))
        place = torch.arange(n * top, device=x.device) - (count.cumsum(0) - count)[mine + 1]
        most = int(count[1:].max())
        there = mine >= 0
        row = torch.where(there, mine * most + place, e * most)
        xg = torch.zeros((e * most + 1, k), dtype=torch.float32, device=x.device)
        xg[row] = x[token[order]]
        gu = torch.bmm(xg[:-1].view(e, most, k), _matrices(s["gate_up"], e, 2 * f, k, None).transpose(1, 2))
        h = gu[..., :f] / (1.0 + torch.exp(-gu[..., :f])) * gu[..., f:]
        y = torch.bmm(h, _matrices(s["down"], e, k, f, None).transpose(1, 2)).view(-1, k)
        y = torch.cat([y, torch.zeros((1, k), device=x.device)])[torch.empty_like(row).index_copy_(0, order, row)]
    w = torch.where(s["expert"] >= 0, s["weight"], 0.0)
    out = (y.view(n, top, k) * w[:, :, None]).sum(1)
    if s["skip"] is not None:
        out = out + s["skip"].float()
    return out.to(dtype)


def _sample(s):
    # 64 bits: sums of a hundred thousand weights, and which of two neighbours a border falls between
    v, order = torch.sort(s["logits"].double(), dim=1, descending=True, stable=True)
    d = v - v[:, :1]
    w = torch.exp(d / s["t"].double()[:, None] if s["t"] is not None else d)
    at = torch.arange(w.shape[1], device=w.device)[None]
    if s["k"] is not None:
        k = s["k"].long()[:, None]
        w = torch.where((at < k) | (k <= 0), w, 0.0)
    c = w.cumsum(1)
    keep = torch.ones_like(w, dtype=torch.bool)
    if s["p"] is not None:
        keep &= (c - w < s["p"].double()[:, None] * c[:, -1:]) | (at == 0)
    if s["m"] is not None:
        keep &= (w >= s["m"].double()[:, None]) | (at == 0)
    w = torch.where(keep, w, 0.0)
    c = w.cumsum(1)
    total = c[:, -1:]
    pick = (c <= s["u"].double()[:, None] * total).sum(1, keepdim=True)
    pick = torch.minimum(pick, (w > 0).sum(1, keepdim=True) - 1)
    return order.gather(1, pick)[:, 0], (w.gather(1, pick) / total)[:, 0].float()


def run(s):
    if own:
        tq2 = s["tq2"]
        if s["op"] == "route":
            return tq2.moe_route(s["logits"], s["top_k"], sigmoid=s["sigmoid"], normalize=s["normalize"], scale=s["scale"])
        if s["op"] == "experts":
            return tq2.moe_swiglu(s["layer"], s["x"], s["expert"], s["weight"], residual=s["skip"], out=s["out"],
                                  workspace=s["workspace"])
        return tq2.sample(s["logits"], s["u"], temperature=s["t"], top_k=s["k"], top_p=s["p"], min_p=s["m"])
    return {"route": _route, "experts": _experts, "sample": _sample}[s["op"]](s)


# ---------------------------------------------------------------------------
# what a pass cannot do without, and what it gives in 64 bits


def work(case):
    size = BYTES[case["dtype"]]
    if case["op"] == "route":
        n = case["tokens"]
        return {"bytes": n * case["experts"] * size + n * case["top_k"] * 8, "flops": 4 * n * case["experts"]}
    if case["op"] == "experts":
        n, e, k, f, top = case["tokens"] - case["padded"], case["experts"], case["width"], case["ffn"], case["top_k"]
        active = e * (1.0 - (1.0 - top / e) ** n)  # experts that have a token, if all are as likely
        rows = case["tokens"] * k * size * (3 if case["residual"] else 2)
        return {"bytes": active * 3 * k * f * 34 / 128 + rows + case["tokens"] * top * 8, "flops": 6 * n * top * k * f}
    return {"bytes": case["rows"] * (case["vocab"] * size + 16), "flops": 4 * case["rows"] * case["vocab"]}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "route":
        l64 = s["logits"].double()
        got = torch.full((case["tokens"], case["top_k"]), 0, dtype=torch.int32, device="cuda")
        w = torch.zeros(got.shape, dtype=torch.float64, device="cuda")
        score = torch.sigmoid(l64) if case["sigmoid"] else torch.softmax(l64, 1)
        left = l64.clone()
        for j in range(case["top_k"]):
            top = left.amax(1, keepdim=True)
            i = (left == top).to(torch.uint8).argmax(1, keepdim=True)
            got[:, j], w[:, j] = i[:, 0].to(torch.int32), score.gather(1, i)[:, 0]
            left.scatter_(1, i, -math.inf)
        if case["normalize"]:
            w /= w.sum(1, keepdim=True)
        return got, w * case["scale"]
    if case["op"] == "experts":
        e, k, f = case["experts"], case["width"], case["ffn"]

        def matrix(soa, i, rows, cols):
            base, size = i * rows * cols // 4, rows * cols // 4
            q = soa[base:base + size].view(rows, cols // 4)
            c = torch.stack([q >> 2 * j & 3 for j in range(4)], -1).view(rows, cols).double() - 1.0
            at = e * size + i * rows * (cols // 128) * 2
            d = soa[at:at + rows * (cols // 128) * 2].view(torch.float16).double()
            return c * d.view(rows, cols // 128).repeat_interleave(128, 1)

        out = s["skip"].double() if s["skip"] is not None else torch.zeros((case["tokens"], k), dtype=torch.float64, device="cuda")
        x = s["x"].double()
        for i in range(e):
            t, j = (s["expert"] == i).nonzero(as_tuple=True)
            if not t.numel():
                continue
            gu = x[t] @ matrix(s["gate_up"], i, 2 * f, k).T
            y = (torch.nn.functional.silu(gu[:, :f]) * gu[:, f:]) @ matrix(s["down"], i, k, f).T
            out.index_add_(0, t, y * s["weight"][t, j].double()[:, None])
        return out
    tokens, probs = [], []
    for r in range(case["rows"]):
        l64 = s["logits"][r].double().cpu()
        order = torch.argsort(-l64, stable=True)
        z = (l64[order] - l64.max()) / (float(s["t"][r]) if s["t"] is not None else 1.0)
        n = len(z)
        if s["k"] is not None and int(s["k"][r]) > 0:
            n = min(n, int(s["k"][r]))
        w = torch.exp(z[:n])
        if s["p"] is not None:
            target = float(s["p"][r]) * math.fsum(w.tolist())
            n = min(n, max(1, int(torch.searchsorted(w.cumsum(0), target)) + 1))
        if s["m"] is not None:
            n = min(n, max(1, int((w >= float(s["m"][r])).sum())))
        c = w[:n].cumsum(0)
        i = min(n - 1, int(torch.searchsorted(c, float(s["u"][r]) * float(c[-1]), right=True)))
        tokens.append(int(order[i]))
        probs.append(float(w[i] / c[-1]))
    return torch.tensor(tokens), torch.tensor(probs, dtype=torch.float64)

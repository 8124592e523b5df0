"""The operators around a ternary transformer's projections, as calls to be timed: rotary positions with several axes,
appending rotated keys and values to a paged cache, and attention of new tokens over that cache.

``run`` computes them in elementary torch operations, or, where ``own`` is true, through the package.  Lengths and
layouts follow from the case alone; values and the order of the pages follow from the seed.
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
        # image model, joint attention: q, k, v of one fused projection (token-major) to the head-major operands of the
        # attention; 512 text tokens and a 64 x 64 latent, four axes of 16 pairs
        dict(name="rope image q k v", op="rope", tokens=4608, heads=24, kv_heads=24, dim=128, pairs=64, axes=4,
             interleaved=True, dtype="f32", out_dtype="f32", to="heads", with_v=True, inverse=False, far=0),
        # video model, gradient: head-major gradients of q and k back to the projection's layout, time x height x width
        dict(name="rope video gradient", op="rope", tokens=14040, heads=12, kv_heads=12, dim=128, pairs=64, axes=3,
             interleaved=False, dtype="bf16", out_dtype="bf16", to="tokens", with_v=False, inverse=True, far=0),
        # a caption's 77 tokens, narrow heads that rotate only partly: launch latency
        dict(name="rope caption", op="rope", tokens=77, heads=5, kv_heads=5, dim=80, pairs=31, axes=2,
             interleaved=False, dtype="f16", out_dtype="f16", to="tokens", with_v=False, inverse=False, far=0),
        # one token of one conversation, far into a long context: launch latency
        dict(name="append one token", op="append", seqs=1, q_lo=1, q_hi=1, kv_lo=99_001, kv_hi=99_001, heads=16,
             kv_heads=2, dim=64, pairs=32, axes=1, interleaved=False, dtype="f32", cache="f16", page=16, order="slots"),
        # decoding step of a batch
        dict(name="append decode batch", op="append", seqs=64, q_lo=1, q_hi=1, kv_lo=37, kv_hi=4096, heads=32,
             kv_heads=8, dim=128, pairs=64, axes=1, interleaved=False, dtype="f32", cache="bf16", page=16,
             order="slots"),
        # ragged prompts with image parts (three axes), a cache whose heads lie outside its slots
        dict(name="append prompts", op="append", seqs=5, q_lo=301, q_hi=8192, kv_lo=301, kv_hi=8192, heads=32,
             kv_heads=8, dim=128, pairs=64, axes=3, interleaved=False, dtype="bf16", cache="bf16", page=64,
             order="heads"),
        # one conversation's next token, short context: launch latency
        dict(name="attend one short", op="attend", seqs=1, q_lo=1, q_hi=1, kv_lo=301, kv_hi=301, heads=32, kv_heads=8,
             dim=128, cache="f16", out_dtype="f16", page=16, order="slots", window=0, causal=True),
        # decoding step of a batch with very different lengths
        dict(name="attend decode batch", op="attend", seqs=64, q_lo=1, q_hi=1, kv_lo=201, kv_hi=8192, heads=32,
             kv_heads=8, dim=128, cache="bf16", out_dtype="bf16", page=16, order="slots", window=0, causal=True),
        # decoding step of one long document, eight query heads a key head
        dict(name="attend decode long", op="attend", seqs=1, q_lo=1, q_hi=1, kv_lo=131_071, kv_hi=131_071, heads=64,
             kv_heads=8, dim=128, cache="bf16", out_dtype="bf16", page=64, order="heads", window=0, causal=True),
        # a chunk of a long prompt against what is cached
        dict(name="attend chunk", op="attend", seqs=1, q_lo=512, q_hi=512, kv_lo=32_768, kv_hi=32_768, heads=32,
             kv_heads=8, dim=128, cache="bf16", out_dtype="bf16", page=64, order="slots", window=0, causal=True),
        # ragged whole prompts
        dict(name="attend prompts", op="attend", seqs=6, q_lo=90, q_hi=4096, kv_lo=90, kv_hi=4096, heads=32,
             kv_heads=8, dim=128, cache="f16", out_dtype="f16", page=16, order="slots", window=0, causal=True),
        # a few drafted tokens per sequence to be verified, a window, odd groups and pages, f32 towards the next
        # projection
        dict(name="attend drafts", op="attend", seqs=16, q_lo=5, q_hi=5, kv_lo=203, kv_hi=3000, heads=14, kv_heads=2,
             dim=64, cache="f16", out_dtype="f32", page=48, order="slots", window=1024, causal=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend"])
    dim = rng.choice([64, 128, 8 * rng.randint(4, 16)])
    pairs = rng.choice([dim // 2, dim // 2, dim // 4, rng.randint(1, dim // 2)])
    interleaved = rng.random() < 0.5
    kv_heads = rng.choice([1, 2, 4, 8, rng.randint(1, 10)])
    heads = kv_heads * rng.choice([1, 2, 4, 4, 8, rng.randint(1, 8)])
    if op == "rope":
        same = rng.random() < 0.5
        dtype = rng.choice(["f32", "f16", "bf16"])
        return dict(op=op, tokens=_log(rng, 1, 12_000), heads=min(heads, 24), kv_heads=min(kv_heads, 24), dim=dim,
                    pairs=pairs, axes=rng.randint(1, 4), interleaved=interleaved, dtype=dtype,
                    out_dtype=dtype if same else rng.choice(["f32", "f16", "bf16"]),
                    to=rng.choice(["heads", "tokens"]), with_v=rng.random() < 0.5, inverse=rng.random() < 0.3,
                    far=_log(rng, 1, 1 << 20))
    page = rng.choice([16, 16, 32, 64, 128, rng.randint(1, 100)])
    order = rng.choice(["slots", "heads"])
    seqs = _log(rng, 1, 64)
    if op == "append":
        q_hi = _log(rng, 1, 8192 // seqs)
        kv_hi = q_hi + _log(rng, 1, 4096)
        return dict(op=op, seqs=seqs, q_lo=_log(rng, 1, q_hi), q_hi=q_hi, kv_lo=rng.randint(1, 2) * q_hi,
                    kv_hi=max(kv_hi, 2 * q_hi), heads=min(heads, 32), kv_heads=kv_heads, dim=dim, pairs=pairs,
                    axes=rng.randint(1, 3), interleaved=interleaved, dtype=rng.choice(["f32", "f16", "bf16"]),
                    cache=rng.choice(["f16", "bf16"]), page=page, order=order)
    kv_hi = _log(rng, 1, 131_072 // seqs)
    q_hi = min(kv_hi, _log(rng, 1, max(1, 4096 // seqs)))
    while seqs * q_hi * kv_hi > 1 << 24:
        q_hi = max(1, q_hi // 2)
    cache = rng.choice(["f16", "bf16"])
    return dict(op=op, seqs=seqs, q_lo=_log(rng, 1, q_hi), q_hi=q_hi, kv_lo=_log(rng, 1, kv_hi), kv_hi=kv_hi,
                heads=min(heads, 8 * kv_heads), kv_heads=kv_heads, dim=dim, cache=cache,
                out_dtype=rng.choice([cache, cache, "f32"]), page=page, order=order,
                window=rng.choice([0, 0, 0, _log(rng, 1, 4096)]), causal=rng.random() < 0.85)


def _spread(n, lo, hi, shift):
    """n lengths from lo to hi, even over their logarithm, in an irregular order; the longest is hi."""
    got = [int(round(lo * (hi / lo) ** ((i * 0.6180339887498949 + shift) % 1.0))) for i in range(n)]
    got[n // 2] = hi
    return got


def _lengths(case):
    """(new tokens, keys after the step) of each sequence; never fewer keys than new tokens."""
    q = _spread(case["seqs"], case["q_lo"], case["q_hi"], 0.31)
    kv = _spread(case["seqs"], case["kv_lo"], case["kv_hi"], 0.31)
    return q, [max(a, b) for a, b in zip(q, kv)]


# ---------------------------------------------------------------------------
# what a user's program has in hand


def _rng(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(gen, shape, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _frequencies(case):
    """inv_freq [pairs] in 64 bits and the axis of each pair: consecutive sections, the lowest frequencies last."""
    pairs, axes = case["pairs"], case["axes"]
    axis = torch.tensor([i * axes // pairs for i in range(pairs)], dtype=torch.int64)
    base = 10_000.0 if axes > 1 else 1_000_000.0
    inv_freq = torch.tensor([base ** (-i / pairs) for i in range(pairs)], dtype=torch.float64)
    return inv_freq, axis


def _grid(tokens, axes, far):
    """Positions of text followed by a grid: [tokens, axes]."""
    t = torch.arange(tokens, device="cuda")
    text = tokens // 9
    side = max(1, math.isqrt(max(1, tokens - text)))
    g = t - text
    cols = [torch.where(g < 0, t, text + g // (side * side) if axes > 2 else text + g // side)]
    if axes > 1:
        cols.append(torch.where(g < 0, t, text + g // side % side))
    if axes > 2:
        cols.append(torch.where(g < 0, t, text + g % side))
    if axes > 3:
        cols.append(torch.where(g < 0, t, 0 * t))
    return torch.stack(cols, 1).contiguous() + far


def _pages(case, gen, state):
    """A cache in use, its pages in the order of the seed: [pages, page, heads, dim] views, the batch's tables."""
    q_len, kv_len = _lengths(case)
    page = case["page"]
    need = [-(-n // page) for n in kv_len]
    total = sum(need) + 3
    shape = (total, page, case["kv_heads"], case["dim"])
    dtype = DTYPES[case["cache"]]

    def pool():
        if case["order"] == "slots":
            return _normal(gen, shape, dtype)
        return _normal(gen, (shape[0], shape[2], shape[1], shape[3]), dtype).transpose(1, 2)

    state["k_cache"], state["v_cache"] = pool(), pool()
    order = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((case["seqs"], max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    starts = [0]
    for n in q_len:
        starts.append(starts[-1] + n)
    state["page_table"] = table
    state["q_start"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    state["kv_len"] = torch.tensor(kv_len, dtype=torch.int32, device="cuda")
    state["tokens"], state["max_q"], state["max_kv"] = starts[-1], max(q_len), max(kv_len)
    return order, kv_len, need


def prepare(case, seed):
    gen = _rng(seed)
    s = dict(case)
    dim = case["dim"]
    if case["op"] == "rope":
        n, dtype, out_dtype = case["tokens"], DTYPES[case["dtype"]], DTYPES[case["out_dtype"]]
        counts = [case["heads"], case["kv_heads"]] + ([case["kv_heads"]] if case["with_v"] else [])

        def rows(h, width, t):  # the slices of one fused projection, [tokens, heads, dim] each
            return [x.unflatten(-1, (-1, dim)) for x in t.split([k * dim for k in h], dim=-1)]

        def heads(h, make):  # contiguous [heads, tokens, dim], seen as [tokens, heads, dim]
            return [make((k, n, dim)).transpose(0, 1) for k in h]

        if case["to"] == "heads":
            s["x"] = rows(counts, dim, _normal(gen, (n, sum(counts) * dim), dtype))
            s["out"] = heads(counts, lambda shape: torch.empty(shape, dtype=out_dtype, device="cuda"))
        else:
            s["x"] = heads(counts, lambda shape: _normal(gen, shape, dtype))
            s["out"] = rows(counts, dim, torch.empty((n, sum(counts) * dim), dtype=out_dtype, device="cuda"))
        s["positions"] = _grid(n, case["axes"], case["far"])
    else:
        order, kv_len, need = _pages(case, gen, s)
        if case["op"] == "append":
            dtype = DTYPES[case["dtype"]]
            h, g = case["heads"], case["kv_heads"]
            fused = _normal(gen, (s["tokens"], (h + 2 * g) * dim), dtype)
            s["q"], s["k"], s["v"] = [x.unflatten(-1, (-1, dim)) for x in fused.split([h * dim, g * dim, g * dim], -1)]
            s["q_out"] = torch.empty((s["tokens"], h, dim), dtype=DTYPES[case["cache"]], device="cuda")
            where = _places(s["q_start"], s["kv_len"], s["tokens"])[1]
            s["positions"] = None if case["axes"] == 1 else torch.stack(
                [where // (1, 3, 2)[a] + a for a in range(case["axes"])], 1).contiguous()
        else:
            # heads attend more or less sharply; the slots past each sequence's end hold whatever was there
            sharp = torch.linspace(0.5, 4.0, case["heads"], device="cuda")[None, :, None]
            s["q"] = (torch.randn((s["tokens"], case["heads"], dim), generator=gen, device="cuda") * sharp).to(
                DTYPES[case["cache"]])
            s["out"] = torch.empty((s["tokens"], case["heads"], dim), dtype=DTYPES[case["out_dtype"]], device="cuda")
            at = 0
            for b, n in enumerate(need):
                last = order[at + n - 1].long()
                for c in (s["k_cache"], s["v_cache"]):
                    c[last, kv_len[b] - (n - 1) * case["page"]:] = float("nan")
                at += n
    if case["op"] != "attend":
        inv_freq, axis = _frequencies(case)
        s["inv_freq"], s["axis"] = inv_freq.cuda(), axis.cuda()
    if own:  # the handles that such a program makes once and keeps: they hold shapes and pointers, and the rope's table
        import dit_tq2_g128_gb300 as tq2
        s["tq2"] = tq2
        if case["op"] != "attend":
            s["rope"] = tq2.Rope(inv_freq, axis, axes=case["axes"], interleaved=case["interleaved"])
        if case["op"] != "rope":
            s["cache_handle"] = tq2.KVCache(s["k_cache"], s["v_cache"])
            s["batch_handle"] = tq2.PagedBatch(s["q_start"], s["kv_len"], s["page_table"], tokens=s["tokens"],
                                               max_q=s["max_q"], max_kv=s["max_kv"])
        if case["op"] == "attend":
            s["workspace"] = tq2.attention_paged_workspace(s["q"], s["cache_handle"], s["batch_handle"])
    return s


# ---------------------------------------------------------------------------
# one pass


def _places(q_start, kv_len, tokens):
    """Sequence and key index of each new token."""
    t = torch.arange(tokens, device=q_start.device)
    seq = torch.searchsorted(q_start[1:].contiguous().long(), t, right=True)
    ends = q_start[1:].long()
    return seq, kv_len.long()[seq] - ends[seq] + t


def _rotate(x, angles, pairs, interleaved, inverse):
    """x [tokens, heads, dim] in 32 bits, angles [tokens, pairs] in 64."""
    c, s = angles.cos().float()[:, None, :], angles.sin().float()[:, None, :]
    if inverse:
        s = -s
    out = x.clone()
    if interleaved:
        a, b = x[..., 0:2 * pairs:2], x[..., 1:2 * pairs:2]
        out[..., 0:2 * pairs:2], out[..., 1:2 * pairs:2] = a * c - b * s, a * s + b * c
    else:
        a, b = x[..., :pairs], x[..., pairs:2 * pairs]
        out[..., :pairs], out[..., pairs:2 * pairs] = a * c - b * s, a * s + b * c
    return out


def _plain_rope(s):
    angles = s["positions"][:, s["axis"]].double() * s["inv_freq"]
    x = [t.float() for t in s["x"]]
    got = [_rotate(t, angles, s["pairs"], s["interleaved"], s["inverse"]) for t in x[:2]] + x[2:]
    return [t.to(DTYPES[s["out_dtype"]]) for t in got]


def _plain_append(s):
    seq, key = _places(s["q_start"], s["kv_len"], s["tokens"])
    positions = key[:, None] if s["positions"] is None else s["positions"]
    angles = positions[:, s["axis"]].double() * s["inv_freq"]
    q = _rotate(s["q"].float(), angles, s["pairs"], s["interleaved"], False)
    k = _rotate(s["k"].float(), angles, s["pairs"], s["interleaved"], False)
    dtype = DTYPES[s["cache"]]
    page = s["page_table"][seq, key // s["page"]].long()
    s["k_cache"][page, key % s["page"]] = k.to(dtype)
    s["v_cache"][page, key % s["page"]] = s["v"].to(dtype)
    return [q.to(dtype), s["k_cache"], s["v_cache"]]


def _plain_attend(s):
    q, table, kv_len, starts = s["q"], s["page_table"].long().clamp(min=0), s["kv_len"].long(), s["q_start"].long()
    seqs, group, dim = s["seqs"], s["heads"] // s["kv_heads"], s["dim"]
    keys = table.shape[1] * s["page"]
    j = torch.arange(keys, device=q.device)
    held = j[None, :] < kv_len[:, None]
    k = s["k_cache"][table].flatten(1, 2).float()  # [seqs, keys, kv heads, dim]
    v = s["v_cache"][table].flatten(1, 2).float()
    v = torch.where(held[:, :, None, None], v, 0.0)
    i = torch.arange(s["max_q"], device=q.device)
    rows = (starts[:-1, None] + i).clamp(max=s["tokens"] - 1)
    pos = kv_len[:, None] - (starts[1:] - starts[:-1])[:, None] + i  # [seqs, max_q]
    sees = held[:, None, :].expand(seqs, s["max_q"], keys)
    if s["causal"]:
        sees = sees & (j[None, None, :] <= pos[:, :, None])
    if s["window"]:
        sees = sees & (j[None, None, :] > pos[:, :, None] - s["window"])
    qs = q[rows].float().unflatten(2, (-1, group)).permute(0, 2, 3, 1, 4)  # [seqs, kv heads, group, max_q, dim]
    scores = qs.flatten(2, 3) @ k.permute(0, 2, 3, 1) * (1.0 / math.sqrt(dim))
    scores = scores.unflatten(2, (group, -1)).masked_fill_(~sees[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = scores.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ v.permute(0, 2, 1, 3)).unflatten(2, (group, -1))
    o = torch.where(total > 0, o / total, 0.0).permute(0, 3, 1, 2, 4).flatten(2, 3)  # [seqs, max_q, heads, dim]
    seq = torch.searchsorted(starts[1:].contiguous(), torch.arange(s["tokens"], device=q.device), right=True)
    return [o[seq, torch.arange(s["tokens"], device=q.device) - starts[seq]].to(DTYPES[s["out_dtype"]])]


def run(s):
    if not own:
        return {"rope": _plain_rope, "append": _plain_append, "attend": _plain_attend}[s["op"]](s)
    tq2 = s["tq2"]
    if s["op"] == "rope":
        tq2.rope_axes(*s["x"], positions=s["positions"], rope=s["rope"], out=s["out"], inverse=s["inverse"])
        return s["out"]
    if s["op"] == "append":
        tq2.kv_append(s["k"], s["v"], s["cache_handle"], s["batch_handle"], rope=s["rope"], positions=s["positions"],
                      q=s["q"], q_out=s["q_out"])
        return [s["q_out"], s["k_cache"], s["v_cache"]]
    return [tq2.attention_paged(s["q"], s["cache_handle"], s["batch_handle"], out=s["out"], window=s["window"],
                                causal=s["causal"], workspace=s["workspace"])]


# ---------------------------------------------------------------------------
# what a pass cannot do without


def work(case):
    dim = case["dim"]
    if case["op"] == "rope":
        values = case["tokens"] * dim * (case["heads"] + case["kv_heads"] * (2 if case["with_v"] else 1))
        turned = case["tokens"] * 2 * case["pairs"] * (case["heads"] + case["kv_heads"])
        return {"bytes": values * (BYTES[case["dtype"]] + BYTES[case["out_dtype"]]) + 8 * case["tokens"] * case["axes"],
                "flops": 3 * turned}
    q_len, kv_len = _lengths(case)
    tokens = sum(q_len)
    if case["op"] == "append":
        values = tokens * dim * (case["heads"] + 2 * case["kv_heads"])
        return {"bytes": values * (BYTES[case["dtype"]] + BYTES[case["cache"]])
                + (8 * tokens * case["axes"] if case["axes"] > 1 else 0),
                "flops": 3 * tokens * 2 * case["pairs"] * (case["heads"] + case["kv_heads"])}
    pairs = held = 0
    for n, m in zip(q_len, kv_len):
        first = m - n
        low = max(0, first - case["window"] + 1) if case["window"] else 0
        held += m - low
        if not case["causal"]:
            whole = n * m
            if case["window"]:
                whole -= sum(max(0, first + i - case["window"] + 1) for i in range(n))
            pairs += whole
        elif case["window"]:
            pairs += sum(min(case["window"], first + i + 1) for i in range(n))
        else:
            pairs += n * first + n * (n + 1) // 2
    return {"bytes": held * case["kv_heads"] * dim * 2 * BYTES[case["cache"]]
            + tokens * case["heads"] * dim * (BYTES[case["cache"]] + BYTES[case["out_dtype"]]),
            "flops": 4 * dim * case["heads"] * pairs}


# ---------------------------------------------------------------------------
# the definitions in 64 bits, token by token or sequence by sequence


def _turn(x, positions, inv_freq, axis, interleaved, inverse):
    """Rotation as a product of complex numbers: x [tokens, heads, dim] in 64 bits."""
    n = inv_freq.numel()
    phase = positions.double().index_select(1, axis) * inv_freq
    unit = torch.polar(torch.ones_like(phase), -phase if inverse else phase).unsqueeze(1)
    head, rest = x[..., :2 * n], x[..., 2 * n:]
    first, second = (head[..., ::2], head[..., 1::2]) if interleaved else (head[..., :n], head[..., n:])
    z = torch.complex(first.contiguous(), second.contiguous()) * unit
    turned = torch.stack((z.real, z.imag), -1).flatten(-2) if interleaved else torch.cat((z.real, z.imag), -1)
    return torch.cat((turned, rest), -1)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rope":
        turned = [_turn(x.double(), s["positions"], s["inv_freq"], s["axis"], case["interleaved"], case["inverse"])
                  for x in s["x"][:2]]
        return turned + [x.double() for x in s["x"][2:]]
    q_len, kv_len = _lengths(case)
    tables = s["page_table"].long()
    if case["op"] == "append":
        keys = torch.cat([torch.arange(m - n, m, device="cuda") for n, m in zip(q_len, kv_len)])
        positions = keys.unsqueeze(1) if s["positions"] is None else s["positions"]
        out = _turn(s["q"].double(), positions, s["inv_freq"], s["axis"], case["interleaved"], False)
        k = _turn(s["k"].double(), positions, s["inv_freq"], s["axis"], case["interleaved"], False)
        caches = [s["k_cache"].double(), s["v_cache"].double()]
        at = 0
        for b, (n, m) in enumerate(zip(q_len, kv_len)):
            j = torch.arange(m - n, m, device="cuda")
            p, o = tables[b][j // case["page"]], j % case["page"]
            caches[0][p, o] = k[at:at + n]
            caches[1][p, o] = s["v"][at:at + n].double()
            at += n
        return [out, *caches]
    if work(case)["flops"] > 5e12:
        return None
    group, at, rows = case["heads"] // case["kv_heads"], 0, []
    for b, (n, m) in enumerate(zip(q_len, kv_len)):
        j = torch.arange(m, device="cuda")
        p, o = tables[b][j // case["page"]], j % case["page"]
        k, v = s["k_cache"][p, o].double(), s["v_cache"][p, o].double()
        block = max(1, 50_000_000 // (m * case["heads"]))
        for lo in range(0, n, block):
            hi = min(n, lo + block)
            at_key = torch.arange(m - n + lo, m - n + hi, device="cuda")
            q = s["q"][at + lo:at + hi].double()
            hidden = torch.zeros((hi - lo, m), dtype=torch.bool, device="cuda")
            if case["causal"]:
                hidden |= j > at_key[:, None]
            if case["window"]:
                hidden |= j <= at_key[:, None] - case["window"]
            heads = []
            for h in range(case["heads"]):
                logits = q[:, h] @ k[:, h // group].T / math.sqrt(case["dim"])
                weights = torch.softmax(logits.masked_fill(hidden, -math.inf), -1).nan_to_num(0.0)
                heads.append(weights @ v[:, h // group])
            rows.append(torch.stack(heads, 1))
        at += n
    return [torch.cat(rows)]


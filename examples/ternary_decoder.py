"""A small decoder of ternary layers, served from a paged key/value cache.

Every projection is a TQ2_0_g128 matmul; between them lie the rotary positions, the cache and its attention:

    q, k, v = x Wqkv                         tq2.matmul (GEMV, skinny or tensor-core kernel by the number of tokens)
    cache <- rotated k, v; q rotated         tq2.kv_append
    a = attention of q over the cache        tq2.attention_paged (f32 out, straight into the next projection)
    x += a Wo; x += swiglu(x Wgu) Wd         tq2.matmul, tq2.tq2_gate_up_swiglu
    or, with experts: x += mixture of them   tq2.moe_route (of a ternary router's logits), tq2.moe_swiglu
    the next token of the logits             argmax, or tq2.sample

A batch of prompts of different lengths is read in chunks, then decoded, one token a sequence a step, each
step one replay of a captured graph whose device tables (lengths, tokens) change between replays.  ``joint_tokens``
is the image model's use of the same rotation: q, k and v of one fused projection, rotated by (text, row, column)
positions into the head-major operands of the joint attention.

    python examples/ternary_decoder.py            # prints the continuation and the rate; weights are random
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import dit_tq2_g128_gb300 as tq2  # noqa: E402

PAGE = 16


class TernaryLinear:
    def __init__(self, n, k, gen):
        self.n, self.k = n, k
        w = torch.randn((n, k), device="cuda", generator=gen) * k ** -0.5
        aos = torch.empty(tq2.tq2_soa_bytes(n, k), dtype=torch.uint8, device="cuda")
        self.w = torch.empty_like(aos)
        tq2.tq2_quantize_f32(w, aos, n, k)
        tq2.tq2_reformat_aos_to_soa(aos, self.w, n, k)

    def __call__(self, x, residual=None):
        return tq2.matmul(self.w, x, residual, n=self.n, k=self.k)


def norm(x):
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)


class Decoder:
    def __init__(self, layers=4, heads=8, kv_heads=2, dim=64, ffn=1024, vocab=1024, seed=0, experts=0, top_k=2):
        """experts: how many of ffn features each layer mixes, top_k of them a token (0: one MLP for all)."""
        gen = torch.Generator(device="cuda").manual_seed(seed)
        self.heads, self.kv_heads, self.dim, self.width, self.vocab, self.ffn = heads, kv_heads, dim, heads * dim, vocab, ffn
        self.embed = torch.randn((vocab, self.width), device="cuda", generator=gen)
        rows = (heads + 2 * kv_heads) * dim
        self.experts, self.top_k = experts, top_k
        many = max(1, experts)
        self.layers = [tuple(TernaryLinear(n, k, gen) for n, k in ((rows, self.width), (self.width, self.width),
                                                                  (many * 2 * ffn, self.width), (many * self.width, ffn)))
                       for _ in range(layers)]
        if experts:
            self.routers = [TernaryLinear(experts, self.width, gen) for _ in range(layers)]
            self.mixtures = [tq2.Experts(gate_up.w, down.w, experts=experts, width=self.width, ffn=ffn)
                             for _, _, gate_up, down in self.layers]
        self.head = TernaryLinear(vocab, self.width, gen)
        self.rope = tq2.Rope([10_000.0 ** (-2 * i / dim) for i in range(dim // 2)])

    def new_caches(self, pages, dtype=torch.bfloat16):
        shape = (pages, PAGE, self.kv_heads, self.dim)
        return [tq2.KVCache(torch.zeros(shape, dtype=dtype, device="cuda"), torch.zeros(shape, dtype=dtype, device="cuda"))
                for _ in self.layers]

    def step(self, tokens, caches, batch):
        """Logits [tokens, vocab] of a step's new tokens (int64 on the device), whose keys join the caches."""
        x = self.embed[tokens]
        h, g, d = self.heads, self.kv_heads, self.dim
        for i, ((qkv, out, gate_up, down), cache) in enumerate(zip(self.layers, caches)):
            q, k, v = (t.unflatten(-1, (-1, d)) for t in qkv(norm(x)).split([h * d, g * d, g * d], -1))
            q = tq2.kv_append(k, v, cache, batch, rope=self.rope, q=q)
            a = tq2.attention_paged(q, cache, batch, out=torch.empty((len(x), h, d), device="cuda"))
            x = out(a.view(len(x), -1), x)
            if self.experts:
                y = norm(x)
                expert, weight = tq2.moe_route(self.routers[i](y), self.top_k)
                x = tq2.moe_swiglu(self.mixtures[i], y, expert, weight, residual=x)
                continue
            act = torch.empty((len(x), self.ffn), device="cuda")
            tq2.tq2_gate_up_swiglu(gate_up.w, norm(x), act, len(x), self.ffn, self.width)
            x = down(act, x)
        return self.head(norm(x))


class Sequences:
    """Lengths and pages of a fixed batch, as device tables that steps read."""

    def __init__(self, count, room):
        per = -(-room // PAGE)
        self.count, self.room, self.pages = count, per * PAGE, count * per
        self.table = torch.randperm(self.pages, device="cuda").to(torch.int32).view(count, per)
        self.kv_len = torch.zeros(count, dtype=torch.int32, device="cuda")

    def batch(self, q_len):
        """A step of q_len[b] new tokens each, counted into the lengths."""
        q_len = torch.tensor(q_len, dtype=torch.int32)
        self.kv_len += q_len.cuda()
        starts = torch.cat([torch.zeros(1, dtype=torch.int32), q_len.cumsum(0).to(torch.int32)])
        return tq2.PagedBatch(starts.cuda(), self.kv_len, self.table, tokens=int(starts[-1]), max_q=int(q_len.max()),
                              max_kv=self.room)


def generate(model, prompts, new, chunk=64, sampling=None):
    """Continuation [sequences, new] of prompts (lists of token ids), and a step's milliseconds: greedy, or drawn with the
    filters of ``sampling`` (keyword arguments of tq2.sample)."""

    def choose(logits):
        if sampling is None:
            return logits.argmax(-1)
        return tq2.sample(logits, torch.rand(len(logits), device="cuda"), **sampling)[0]

    seqs = Sequences(len(prompts), max(map(len, prompts)) + new)
    caches = model.new_caches(seqs.pages)
    last = [None] * len(prompts)
    for at in range(0, max(map(len, prompts)), chunk):
        parts = [p[at:at + chunk] for p in prompts]
        logits = model.step(torch.tensor(sum(parts, []), device="cuda"), caches, seqs.batch([len(p) for p in parts]))
        end = 0
        for b, p in enumerate(parts):
            end += len(p)
            if p:
                last[b] = logits[end - 1]
    token = choose(torch.stack(last))
    # decoding: one graph, replayed with the lengths and tokens that the last replay left
    step = seqs.batch([1] * len(prompts))
    out = torch.empty((new, len(prompts)), dtype=torch.int64, device="cuda")
    row = torch.zeros(1, dtype=torch.int64, device="cuda")

    def one():
        out.index_copy_(0, row, token[None])
        token.copy_(choose(model.step(token, caches, step)))
        seqs.kv_len.add_(1)
        row.add_(1)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        one()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        one()
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    for _ in range(new - 1):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    return out.T, begin.elapsed_time(end) / max(1, new - 1)


def joint_tokens(fused, heads, dim, text, side):
    """Joint attention of text tokens and a side x side image: fused [tokens, 3 * heads * dim] f32 of one projection
    (text first) -> [tokens, heads * dim]."""
    tokens = fused.shape[0]
    third = dim // 2 // 3
    axis = [0] * (dim // 2 - 2 * third) + [1] * third + [2] * third
    rope = tq2.Rope([10_000.0 ** (-i / (dim // 2)) for i in range(dim // 2)], axis, axes=3, interleaved=True)
    t = torch.arange(tokens, device="cuda")
    image = t - text
    positions = torch.stack([torch.where(image < 0, t, text + 0 * t), torch.where(image < 0, 0 * t, image // side),
                             torch.where(image < 0, 0 * t, image % side)], 1).contiguous()
    q, k, v = (x.unflatten(-1, (heads, dim)) for x in fused.chunk(3, -1))
    out = [torch.empty((heads, tokens, dim), device="cuda") for _ in range(3)]
    tq2.rope_axes(q, k, v, positions=positions, rope=rope, out=[x.transpose(0, 1) for x in out])
    a = torch.empty((tokens, heads * dim), device="cuda")
    tq2.tq2_attention_f32(*out, a, heads, tokens, dim)
    return a


def main():
    torch.manual_seed(0)
    model = Decoder()
    prompts = [torch.randint(0, model.vocab, (n,)).tolist() for n in (200, 37, 1, 90)]
    tokens, ms = generate(model, prompts, 64)
    for p, row in zip(prompts, tokens.tolist()):
        print(f"{len(p):4d} tokens -> {row[:12]} ...")
    print(f"{ms:.3f} ms a step, {len(prompts) / ms * 1e3:.0f} tokens/s")
    mixture = Decoder(ffn=512, experts=8)
    each = lambda v, t=torch.float32: torch.full((len(prompts),), v, dtype=t, device="cuda")  # noqa: E731
    tokens, ms = generate(mixture, prompts, 64, sampling=dict(temperature=each(0.8), top_k=each(40, torch.int32), top_p=each(0.95)))
    for p, row in zip(prompts, tokens.tolist()):
        print(f"{len(p):4d} tokens -> {row[:12]} ... (8 experts, sampled)")
    print(f"{ms:.3f} ms a step, {len(prompts) / ms * 1e3:.0f} tokens/s")
    print("joint attention:", tuple(joint_tokens(torch.randn(77 + 256, 3 * 4 * 64, device="cuda"), 4, 64, 77, 16).shape))
    assert tq2.tq2_device_status() == tq2.TQ2_OK


if __name__ == "__main__":
    main()

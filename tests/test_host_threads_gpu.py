"""Two host threads, each on a stream of its own, call the same entry point with sizes that need different amounts of shared
memory: what one thread's call asks of a kernel must not fail the other's launch."""

import threading

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def tq2():
    import dit_tq2_g128_gb300 as m
    return m


def at_once(calls, times):
    """Runs each of `calls` (functions of a stream) `times` times in a thread of its own; what they raised."""
    errors, begin = [], threading.Barrier(len(calls))
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()

    def work(call, stream):
        try:
            begin.wait()
            for i in range(times):
                call(stream)
                if i % 64 == 63:
                    stream.synchronize()
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=work, args=a) for a in zip(calls, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return errors


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_sampling_of_two_vocabularies(tq2, dtype):
    torch_type, kind = {"f32": (torch.float32, tq2.TQ2_F32), "bf16": (torch.bfloat16, tq2.TQ2_BF16)}[dtype]
    calls, results = [], []
    for rows, vocab in ((1, 200_000), (2, 32_000), (1, 3000), (1, 260_000)):
        gen = torch.Generator(device="cuda").manual_seed(vocab)
        x = torch.randn((rows, vocab), device="cuda", generator=gen).to(torch_type)
        u, k = torch.rand(rows, device="cuda", generator=gen), torch.full((rows,), 30, dtype=torch.int32, device="cuda")
        want = tq2.sample(x, u, top_k=k)
        out = torch.empty_like(want[0]), torch.empty_like(want[1])
        results.append((want, out, x, u, k))
        # (the C entry point with its arguments at hand, so that most of a call is spent in it)
        at = x.data_ptr(), kind, vocab, u.data_ptr(), tq2.tq2_sampling(top_k=k), out[0].data_ptr(), out[1].data_ptr(), rows, vocab

        def call(stream, at=at):
            status = tq2.lib.tq2_sample(*at, stream.cuda_stream)
            if status:
                raise tq2.TQ2Error(status, "tq2_sample")

        calls.append(call)
    assert at_once(calls, 5000) == []
    for want, out, *_ in results:
        assert torch.equal(want[0], out[0]) and torch.equal(want[1], out[1])


def products(tq2, kernel, shapes, times):
    """The same kernel's products of several shapes (m, n, k) at once."""
    calls, results = [], []
    for m, n, k in shapes:
        gen = torch.Generator(device="cuda").manual_seed(n + k)
        w = torch.randint(0, 256, (tq2.tq2_soa_bytes(n, k),), dtype=torch.uint8, device="cuda", generator=gen)
        w[n * k // 4:].view(torch.float16).uniform_(0.5 * k ** -0.5, 1.5 * k ** -0.5, generator=gen)
        x = torch.randn((m, k), device="cuda", generator=gen)
        want, out = (torch.empty((m, n), device="cuda") for _ in range(2))
        call = lambda s, o, w=w, x=x, m=m, n=n, k=k: tq2.tq2_gemm_with(kernel, w, x, None, o, m, n, k, stream=s)  # noqa: E731
        call(None, want)
        results.append((want, out))
        calls.append(lambda s, call=call, out=out: call(s, out))
    assert at_once(calls, times) == []
    for want, out in results:
        assert torch.equal(want, out)


# (the pairs share a kernel: as many rows a stage)
@pytest.mark.parametrize("shapes", [[(1, 12_288, 4096), (1, 4096, 4096)], [(1, 12_288, 5120), (1, 12_288, 1024)]])
def test_gemv_of_two_sizes(tq2, shapes):
    products(tq2, tq2.TQ2_KERNEL_GEMV, shapes, 2000)


def test_small_products_of_two_lengths(tq2):
    products(tq2, tq2.TQ2_KERNEL_SKINNY, [(4, 7296, 262_144), (4, 7296, 131_072)], 200)


def test_skinny_products_of_two_sizes(tq2):
    products(tq2, tq2.TQ2_KERNEL_SKINNY_MMA, [(8, 4096, 4096), (8, 1024, 1024), (7, 9728, 8192)], 2000)


def first_calls(tq2):
    """Functions of an output, one for each kernel that copies by tensor maps, and the outputs' shapes and types."""
    gen = torch.Generator(device="cuda").manual_seed(1)

    def weight(n, k):
        w = torch.randint(0, 256, (tq2.tq2_soa_bytes(n, k),), dtype=torch.uint8, device="cuda", generator=gen)
        w[n * k // 4:].view(torch.float16).uniform_(0.5 * k ** -0.5, 1.5 * k ** -0.5, generator=gen)
        return w

    w = weight(256, 1024)
    rows = torch.randn((300, 1024), device="cuda", generator=gen)
    ws = torch.empty(tq2.tq2_gemm_workspace_bytes(300, 256, 1024), dtype=torch.uint8, device="cuda")
    heads = torch.randn((3, 2, 70, 64), device="cuda", generator=gen)
    pages = torch.randn((2, 12, 16, 1, 64), device="cuda", generator=gen).to(torch.bfloat16)
    q = torch.randn((140, 4, 64), device="cuda", generator=gen).to(torch.bfloat16)
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.arange(10, dtype=torch.int32, device="cuda")[None]
    cache = tq2.KVCache(pages[0], pages[1])
    batch = {t: tq2.PagedBatch(ints(0, t), ints(140), table, tokens=t, max_q=t, max_kv=140) for t in (1, 140)}
    layer = tq2.Experts(weight(512, 256), weight(512, 128), experts=2, width=256, ffn=128)
    expert, scale = torch.zeros((9, 1), dtype=torch.int32, device="cuda"), torch.ones((9, 1), device="cuda")
    moe_ws = tq2.moe_swiglu_workspace(layer, 9, 1, torch.float32)
    s = 0  # (the default stream, by its handle)
    f32, bf16 = torch.float32, torch.bfloat16
    return {
        "gemv": (lambda o: tq2.tq2_gemv(w, rows, None, o, 256, 1024, stream=s), (256,), f32),
        "skinny": (lambda o: tq2.tq2_gemm_with(tq2.TQ2_KERNEL_SKINNY_MMA, w, rows, None, o, 8, 256, 1024, stream=s), (8, 256), f32),
        "rows": (lambda o: tq2.tq2_gemm_ws(w, rows, None, o, 300, 256, 1024, ws, ws.numel(), stream=s), (300, 256), f32),
        "joint attention": (lambda o: tq2.tq2_attention_f32(*heads, o, 2, 70, 64, stream=s), (70, 128), f32),
        "paged, few rows": (lambda o: tq2.attention_paged(q[:1], cache, batch[1], out=o, stream=s), (1, 4, 64), bf16),
        "paged, many rows": (lambda o: tq2.attention_paged(q, cache, batch[140], out=o, stream=s), (140, 4, 64), bf16),
        "experts": (lambda o: tq2.moe_swiglu(layer, rows.view(-1, 256)[:9], expert, scale, out=o, workspace=moe_ws, stream=s), (9, 256), f32),
    }


@pytest.mark.parametrize("name", ["gemv", "skinny", "rows", "joint attention", "paged, few rows", "paged, many rows", "experts"])
def test_the_first_call_of_a_host_thread(tq2, name):
    """A thread that has made no CUDA call yet gets what others get."""
    call, shape, dtype = first_calls(tq2)[name]
    want, got, errors = torch.empty(shape, dtype=dtype, device="cuda"), torch.empty(shape, dtype=dtype, device="cuda"), []

    def work():
        try:
            call(got)
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    call(want)
    torch.cuda.synchronize()
    thread = threading.Thread(target=work)
    thread.start()
    thread.join()
    torch.cuda.synchronize()
    assert errors == []
    assert torch.equal(want, got)

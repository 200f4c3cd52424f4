"""Captured calls with the default workspace: a graph's scratch is its own, whatever calls came
before on the stream it was captured on and whatever larger ones come after."""
import pytest

torch = pytest.importorskip("torch")
import kv_ref as R  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sv():
    import __graft_entry__
    __graft_entry__.build()
    import speculative_decoding_verification_59_gb300 as m
    return m


def attention(sv, B, N, Hq, H, longest):
    g = torch.Generator(device="cuda").manual_seed(N)
    cache = sv.KVCache(*R.make_cache_on_gpu(N, B, longest + N, 16, H, 128))
    q = (torch.randn((B, N, Hq, 128), generator=g, device="cuda") * 1.5).to(torch.bfloat16)
    ctx = torch.full((B,), longest, dtype=torch.int32, device="cuda")
    need = sv.load_library().spec_attention_workspace_size(B, N, Hq, H, 128)
    return (lambda: sv.paged_attention(q, cache, ctx, lse=True)), need


def logprobs(sv, rows, V, K):
    g = torch.Generator(device="cuda").manual_seed(rows)
    z = torch.randn((rows, V), generator=g, device="cuda") * 3
    tok = torch.randint(0, V, (rows,), generator=g, device="cuda").to(torch.int32)
    need = sv.load_library().spec_logprobs_workspace_size(rows, V, K)
    return (lambda: sv.token_logprobs(z, tok, K)), need


@pytest.mark.parametrize("kind", ["attention", "logprobs"])
def test_a_larger_call_after_the_capture(sv, kind):
    """A small call is made and then captured on one stream, a larger one made there after that.
    What the larger one gave back to the allocator is handed out and filled: replays give the
    same results and leave the fill alone."""
    if kind == "attention":
        small, need = attention(sv, 2, 1, 8, 2, 3000)
        large, more = attention(sv, 4, 36, 8, 2, 2000)
    else:
        small, need = logprobs(sv, 3, 151936, 4)
        large, more = logprobs(sv, 64, 151936, 4)
    assert more > need
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        want = [t.clone() for t in small()]
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            held = small()
        big = [t.clone() for t in large()]
        s.synchronize()
        fills = [torch.full((n,), 171, dtype=torch.uint8, device="cuda") for n in (need, need, 256, need + 512, more) for _ in range(3)]
        for _ in range(3):
            graph.replay()
        s.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want))
        assert all((f == 171).all() for f in fills)
        assert all(torch.equal(a, b) for a, b in zip(large(), big))
        s.synchronize()


@pytest.mark.parametrize("kind", ["attention", "logprobs"])
def test_replays_beside_calls_on_the_stream_of_the_capture(sv, kind):
    """A graph replayed on one stream while the same kind of call runs on the stream it was captured
    on: neither touches the other's scratch."""
    make = (lambda n: attention(sv, 2 + n, 2 + n, 8, 2, 3000 - n)) if kind == "attention" else (lambda n: logprobs(sv, 20 + n, 50257, 3))
    (first, _), (second, _) = make(0), make(1)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(a):
        second()                                               # (leaves a workspace that is large enough)
        want = [t.clone() for t in first()]
        other = [t.clone() for t in second()]
        a.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=a):
            held = first()
    torch.cuda.synchronize()
    got = []
    for _ in range(30):
        with torch.cuda.stream(b):
            graph.replay()
        with torch.cuda.stream(a):
            got.append(second())
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(held, want))
    for r in got:
        assert all(torch.equal(x, y) for x, y in zip(r, other))

"""What the native marshalling of the cache, attention and log-probability calls leaves behind and
takes: the current device and stream, strides of single rows, host threads on one stream and on
several."""
import threading

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


def current():
    return torch.cuda.current_device(), [torch.cuda.current_stream(d).cuda_stream for d in range(torch.cuda.device_count())]


def every_call(sv, device, **kw):
    """One of each call on tensors of a device."""
    with torch.cuda.device(device):
        cache = sv.KVCache(*R.make_cache_on_gpu(1, 2, 64, 16, 2, 64))
        k = torch.randn((2, 3, 2, 64), device="cuda").to(torch.bfloat16)
        ctx = torch.tensor([10, 20], dtype=torch.int32, device="cuda")
        path = torch.tensor([[2, 0, 0], [1, 2, 0]], dtype=torch.int32, device="cuda")
        z = torch.randn((4, 100), device="cuda")
        torch.cuda.synchronize()
    return (lambda: sv.kv_append(cache, k, k, k, ctx, **kw), lambda: sv.paged_attention(k, cache, ctx, **kw),
            lambda: sv.kv_compact(cache, ctx, path, ctx * 0 + 1, **kw), lambda: sv.kv_read(cache, 9, **kw),
            lambda: sv.token_logprobs(z, torch.zeros(4, dtype=torch.int32, device=z.device), 2, **kw))


def test_the_current_device_and_stream_stay(sv):
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(other):
        before = current()
        for kw in ({}, {"stream": side}):
            for f in every_call(sv, 0, **kw):
                f()
                assert current() == before
    torch.cuda.synchronize()


@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="tensors of another device than the current one")
def test_the_current_device_stays_when_the_tensors_are_anothers(sv):
    side = torch.cuda.Stream(device=1)
    with torch.cuda.device(0):
        before = current()
        for kw in ({}, {"stream": side}):
            for f in every_call(sv, 1, **kw):
                f()
                assert current() == before
    torch.cuda.synchronize(1)


def test_one_token_has_no_stride(sv):
    """A single token's row cut from a buffer whose rows are of any length."""
    cache = sv.KVCache(*R.make_cache_on_gpu(5, 1, 64, 16, 2, 64))
    ctx = torch.tensor([7], dtype=torch.int32, device="cuda")
    buffer = torch.randn(3, 1, 8 * 64 + 3, device="cuda").to(torch.bfloat16)
    q, k, v = buffer[:, :, :512].view(3, 1, 8, 64)[:1].split((4, 2, 2), 2)
    assert q.stride(0) % 8
    prepared = sv.kv_append(cache, q, k, v, ctx)
    assert torch.equal(prepared, q)
    got = [t[0, 7] for t in sv.kv_read(cache, 8)]
    assert torch.equal(got[0], k[0, 0]) and torch.equal(got[1], v[0, 0])
    assert torch.equal(sv.paged_attention(q, cache, ctx), sv.paged_attention(q.contiguous(), cache, ctx))
    with pytest.raises(sv.SpecVerifyError):                    # two such rows are as far apart as they say
        two = torch.randn(2, 1, 8 * 64 + 3, device="cuda").to(torch.bfloat16)[:, :, :256].view(2, 1, 4, 64)
        sv.paged_attention(two, sv.KVCache(cache.k, cache.v, cache.block_table.repeat(2, 1)), ctx.repeat(2))


@pytest.mark.parametrize("shared", [False, True])
def test_host_threads(sv, shared):
    """Six threads make their calls at once, with the default workspaces: each on a stream of its own,
    or all on one.  Every result is that of the call made alone."""
    def job(i):
        g = torch.Generator(device="cuda").manual_seed(i)
        N, longest = 1 + 5 * (i % 3), 700 + 900 * (i % 4)
        cache = sv.KVCache(*R.make_cache_on_gpu(i, 2, longest + N, 16, 2, 128, fp8=i % 2 == 1))
        q = torch.randn((2, N, 8, 128), generator=g, device="cuda").to(torch.bfloat16)
        k, v = (torch.randn((2, N, 2, 128), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
        ctx = torch.tensor([longest, 40 + i], dtype=torch.int32, device="cuda")
        z = torch.randn((20 + 30 * i, 30011), generator=g, device="cuda") * 3
        tok = torch.randint(0, 30011, (len(z),), generator=g, device="cuda").to(torch.int32)

        def run(stream, reps):
            out = []
            for _ in range(reps):
                p = sv.kv_append(cache, q, k, v, ctx, stream=stream)
                out.append((*sv.paged_attention(p, cache, ctx, lse=True, stream=stream), *sv.kv_read(cache, 60, stream=stream),
                            *sv.token_logprobs(z, tok, 4, stream=stream)))
            stream.synchronize()
            return out
        return run
    jobs = [job(i) for i in range(6)]
    torch.cuda.synchronize()
    one = torch.cuda.Stream()
    got, wrong = [None] * 6, []

    def worker(i):
        try:
            got[i] = jobs[i](one if shared else torch.cuda.Stream(), 25)
        except Exception as e:                                 # reported below
            wrong.append((i, repr(e)))
    threads = [threading.Thread(target=worker, args=(i,)) for i in range(6)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    torch.cuda.synchronize()
    for i in range(6):
        alone = jobs[i](torch.cuda.Stream(), 1)[0]
        torch.cuda.synchronize()
        for r in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(r, alone))


def test_scales_of_a_cache_are_tensors(sv):
    k, v, table, ks, vs = R.make_cache_on_gpu(6, 1, 32, 16, 2, 64, fp8=True)
    for bad in (0.5, [1.0], ks.cpu().numpy()):
        with pytest.raises(TypeError, match="k_scale must be a torch tensor"):
            sv.KVCache(k, v, table, bad, vs)
        with pytest.raises(TypeError, match="v_scale must be a torch tensor"):
            sv.KVCache(k, v, table, ks, bad)
    for bad in (ks.double(), ks[:, :, :1], ks.cpu()):
        with pytest.raises(ValueError, match="k_scale must be float32"):
            sv.KVCache(k, v, table, bad, vs)

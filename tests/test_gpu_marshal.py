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

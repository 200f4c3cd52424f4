"""Host-side checks of the cache, attention and log-probability calls that need no GPU: every
refusal comes back before the device is touched (no kernel is launched here)."""
import ctypes
import os

import pytest

import speculative_decoding_verification_59_gb300 as sv

FAKE, WS = 1 << 20, 1 << 24          # aligned addresses that are never dereferenced


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(sv.lib_path()):
        import __graft_entry__
        __graft_entry__.build()
    return sv.load_library()


def cache(**kw):
    a = dict(k=FAKE, v=FAKE, k_scale=None, v_scale=None, block_table=FAKE, error=None, page_stride=16 * 256,
             token_stride=256, head_stride=128, layer_stride=0, scale_page_stride=0, scale_token_stride=0,
             scale_head_stride=0, scale_layer_stride=0, dtype=sv.SPEC_DTYPE_BF16, layers=1, num_pages=10, page_size=16,
             max_pages=4, kv_heads=2, head_dim=128)
    a.update(kw)
    return sv.KVCacheStruct(*(a[n] for n, _ in sv.KVCacheStruct._fields_))


BAD_CACHES = [
    (dict(dtype=sv.SPEC_DTYPE_F32), sv.SPEC_ERR_UNSUPPORTED_DTYPE),
    (dict(k=None), sv.SPEC_ERR_INVALID_ARG),
    (dict(block_table=None), sv.SPEC_ERR_INVALID_ARG),
    (dict(dtype=sv.SPEC_DTYPE_E4M3), sv.SPEC_ERR_INVALID_ARG),                # no scales
    (dict(head_dim=96), sv.SPEC_ERR_INVALID_ARG),
    (dict(page_size=0), sv.SPEC_ERR_INVALID_ARG),
    (dict(max_pages=1 << 28), sv.SPEC_ERR_INVALID_ARG),                       # positions past 31 bits
    (dict(k=FAKE + 8), sv.SPEC_ERR_MISALIGNED),
    (dict(token_stride=260), sv.SPEC_ERR_MISALIGNED),
]


def attend(c, **kw):
    a = dict(q=FAKE, qs=1024, ctx=FAKE, newl=None, par=None, scale=0.1, B=2, N=3, Hq=8, out=FAKE, lse=None, ws=WS, wb=1 << 30)
    a.update(kw)
    return sv.load_library().spec_paged_attention(ctypes.addressof(c) if c else None, a["q"], a["qs"], a["ctx"], a["newl"],
                                                  a["par"], a["scale"], a["B"], a["N"], a["Hq"], a["out"], a["lse"],
                                                  a["ws"], a["wb"], None)


def append(c, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, qs=1024, ks=256, vs=256, qw=None, kw=None, eps=1e-6, rope=FAKE, rows=100, rot=128,
             inter=0, ctx=FAKE, newl=None, pos=None, B=2, N=3, Hq=8, out=FAKE)
    a.update(kw)
    return sv.load_library().spec_kv_append(ctypes.addressof(c) if c else None, *(a[n] for n in a), None)


def read(c, **kw):
    a = dict(starts=None, counts=None, B=2, T=5, dt=sv.SPEC_DTYPE_BF16, k=FAKE, v=FAKE)
    a.update(kw)
    return sv.load_library().spec_kv_read(ctypes.addressof(c) if c else None, *(a[n] for n in a), None)


def compact(c, **kw):
    a = dict(ctx=FAKE, path=FAKE, acc=FAKE, B=2, N=5)
    a.update(kw)
    return sv.load_library().spec_kv_compact(ctypes.addressof(c) if c else None, *(a[n] for n in a), None)


@pytest.mark.parametrize("change,status", BAD_CACHES)
def test_every_call_refuses_a_bad_cache(lib, change, status):
    for call in (attend, append, read, compact):
        assert call(cache(**change)) == status
        assert call(None) == sv.SPEC_ERR_INVALID_ARG
        assert call(cache(**change), B=0) == sv.SPEC_OK


def test_attention_refusals(lib):
    c = cache()
    inv, mis = sv.SPEC_ERR_INVALID_ARG, sv.SPEC_ERR_MISALIGNED
    for kw, status in ((dict(B=-1), inv), (dict(N=0), inv), (dict(N=258), inv), (dict(N=65, par=FAKE), inv),
                       (dict(scale=float("inf")), inv), (dict(scale=float("nan")), inv), (dict(Hq=7), inv), (dict(Hq=0), inv),
                       (dict(Hq=130), inv), (dict(q=None), inv), (dict(ctx=None), inv), (dict(out=None), inv), (dict(ws=None), inv),
                       (dict(q=FAKE + 2), mis), (dict(qs=1025), mis), (dict(out=FAKE + 8), mis), (dict(ws=WS + 16), mis),
                       (dict(wb=1000), sv.SPEC_ERR_WORKSPACE_TOO_SMALL)):
        assert attend(c, **kw) == status, kw
    assert lib.spec_attention_workspace_size(1, 1, 7, 2, 128) == 0
    assert lib.spec_attention_workspace_size(1, 1, 8, 2, 96) == 0
    assert lib.spec_attention_workspace_size(1, 258, 8, 2, 128) == 0
    assert 0 < lib.spec_attention_workspace_size(1, 1, 8, 2, 128) <= lib.spec_attention_workspace_size(64, 8, 8, 2, 128)


def test_append_refusals(lib):
    c = cache()
    inv, mis = sv.SPEC_ERR_INVALID_ARG, sv.SPEC_ERR_MISALIGNED
    for kw, status in ((dict(B=-1), inv), (dict(N=0), inv), (dict(Hq=-1), inv), (dict(k=None), inv), (dict(v=None), inv),
                       (dict(q=None), inv), (dict(out=None), inv), (dict(ctx=None), inv), (dict(rope=None), inv), (dict(rows=0), inv),
                       (dict(rot=24), inv), (dict(rot=144), inv), (dict(rot=-16), inv), (dict(kw=FAKE, eps=-1.0), inv),
                       (dict(kw=FAKE, eps=float("nan")), inv), (dict(q=FAKE + 2), mis), (dict(ks=257), mis),
                       (dict(v=FAKE + 8), mis), (dict(rope=FAKE + 4), mis), (dict(qw=FAKE + 2), mis), (dict(B=1 << 20, N=1 << 10), inv)):
        assert append(c, **kw) == status, kw


def test_read_and_compact_refusals(lib):
    c = cache()
    inv, mis = sv.SPEC_ERR_INVALID_ARG, sv.SPEC_ERR_MISALIGNED
    for kw, status in ((dict(B=-1), inv), (dict(T=-1), inv), (dict(k=None), inv), (dict(v=None), inv), (dict(B=70000), inv),
                       (dict(dt=2), sv.SPEC_ERR_UNSUPPORTED_DTYPE), (dict(k=FAKE + 8), mis), (dict(T=0), sv.SPEC_OK)):
        assert read(c, **kw) == status, kw
    for kw, status in ((dict(B=-1), inv), (dict(N=0), inv), (dict(N=1025), inv), (dict(path=None), inv), (dict(acc=None), inv),
                       (dict(ctx=None), inv), (dict(B=70000), inv)):
        assert compact(c, **kw) == status, kw


def test_logprobs_refusals(lib):
    f = lib.spec_token_logprobs
    need = lib.spec_logprobs_workspace_size(3, 100, 4)
    ok = dict(z=FAKE, dt=1, tok=FAKE, T=1.0, rows=3, V=100, K=4, lp=FAKE, ent=None, ti=FAKE, tl=FAKE, ws=WS, wb=need)

    def call(**kw):
        a = dict(ok, **kw)
        return f(*(a[n] for n in a), None)
    inv, mis = sv.SPEC_ERR_INVALID_ARG, sv.SPEC_ERR_MISALIGNED
    for kw, status in ((dict(dt=2), sv.SPEC_ERR_UNSUPPORTED_DTYPE), (dict(rows=-1), inv), (dict(V=0), inv), (dict(V=(1 << 24) + 1), inv), (dict(K=9), inv),
                       (dict(K=-1), inv), (dict(T=0.0), inv), (dict(T=float("nan")), inv), (dict(z=None), inv), (dict(tok=None), inv),
                       (dict(lp=None), inv), (dict(ti=None), inv), (dict(tl=None), inv), (dict(ws=None), inv), (dict(z=FAKE + 2), mis),
                       (dict(ws=WS + 8), mis), (dict(wb=need - 1), sv.SPEC_ERR_WORKSPACE_TOO_SMALL), (dict(rows=0), sv.SPEC_OK)):
        assert call(**kw) == status, kw
    assert lib.spec_logprobs_workspace_size(3, 100, 9) == 0 and lib.spec_logprobs_workspace_size(3, 0, 1) == 0


def test_tensor_helpers_refuse_host_tensors():
    torch = pytest.importorskip("torch")
    k = torch.zeros((2, 16, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        sv.KVCache(k, k, torch.zeros((1, 2), dtype=torch.int32))
    with pytest.raises(TypeError, match="torch tensor"):
        sv.KVCache(k.float().numpy(), k, torch.zeros((1, 2), dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        sv.token_logprobs(torch.zeros((2, 10)), torch.zeros(2, dtype=torch.int32))

"""A chunk of a prompt through the cache: the longest chains the calls take, grouped heads, behind
contexts of any length, appended and attended, against the 64-bit forms (tests/kv_ref.py)."""
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


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("N,Hq,H,D,ctx,newl", [
    (257, 8, 2, 128, [0], None),                      # 1028 rows of a cached head
    (257, 4, 1, 128, [900, 0, 3], [257, 200, 1]),
    (256, 4, 1, 128, [130], None),
    (200, 5, 1, 128, [64], [129]),
    (257, 4, 1, 64, [300], None),
    (257, 4, 1, 256, [70], None),
])
def test_chunks(sv, fp8, N, Hq, H, D, ctx, newl):
    g = torch.Generator().manual_seed(N + D)
    B = len(ctx)
    parts = R.make_cache(60, B, max(ctx) + N, 16, H, D, fp8)
    cache = R.on_gpu(sv, parts)
    qkv = torch.randn((B, N, Hq + 2 * H, D), generator=g).to(torch.bfloat16)
    q, k, v = qkv.split((Hq, H, H), 2)
    w = (torch.rand(D, generator=g) + 0.5).to(torch.bfloat16)
    rope = R.rope_table(max(ctx) + N, D)
    c = torch.tensor(ctx, dtype=torch.int32)
    nb = torch.tensor(newl or [N] * B, dtype=torch.int32)
    dq, dk, dv = qkv.cuda().split((Hq, H, H), 2)
    prepared = sv.kv_append(cache, dq, dk, dv, c.cuda(), rope.cuda(), q_weight=w.cuda(), k_weight=w.cuda(), new_lens=nb.cuda())
    out, lse = sv.paged_attention(prepared, cache, c.cuda(), new_lens=nb.cuda(), lse=True)
    assert cache.read_error() == 0
    pos = c[:, None] + torch.arange(N)
    want, mag = R.norm_rope(q, w, rope, pos, 1e-6, False)
    for b in range(B):                                         # queries: fp32 steps, rounded once
        n = int(nb[b])
        assert ((prepared[b, :n].cpu().double() - want[b, :n]).abs()
                <= R.U_BF16 * want[b, :n].abs() + 2 * D * R.U_F32 * mag[b, :n]).all()
    # attention over what the append has written
    held = [None if t is None else t.cpu() for t in (cache.k, cache.v, cache.block_table, cache.k_scale, cache.v_scale)]
    o, l, to, tl = R.attention(prepared.cpu(), *held, c, nb)
    out, lse = out.cpu().double(), lse.cpu().double()
    for b in range(B):
        n = int(nb[b])
        assert ((out[b, :n] - o[b, :n]).abs() <= to[b, :n]).all()
        assert ((lse[b, :n] - l[b, :n]).abs() <= tl[b, :n]).all()
        assert (out[b, n:] == 0).all() and torch.isneginf(lse[b, n:]).all()

"""The cache calls against their 64-bit forms (tests/kv_ref.py): append with head norms,
rotation and quantisation, reading back, and moving a tree's accepted path."""
import math

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


def gather(cache, b, t):
    """Rows at positions t of sequence b as the cache holds them: (k, v) [n, H, D] float64."""
    page = cache.page_size
    pg = cache.block_table[b].long()[t // page]
    both = []
    for x, s in ((cache.k, cache.k_scale), (cache.v, cache.v_scale)):
        y = x.float()[pg, t % page].double()
        both.append((y if s is None else y * s[pg, t % page].double()[..., None]).cpu())
    return both


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B,N,Hq,H,D,page,ctx,rot,inter,norm,fused", [
    (1, 1, 1, 1, 64, 16, [0], 64, False, True, False),
    (1, 1, 32, 8, 128, 16, [777], 128, False, True, True),
    (3, 5, 7, 1, 128, 5, [0, 4, 31], 64, False, True, True),      # odd heads, partial rotation
    (2, 8, 8, 2, 64, 48, [40, 95], 32, True, True, False),
    (2, 3, 6, 3, 256, 16, [13, 200], 256, False, False, True),
    (4, 2, 4, 4, 256, 1, [0, 1, 2, 9], 256, True, True, True),
    (2, 4, 5, 5, 128, 16, [3, 60], 0, False, True, True),         # no rotation
    (2, 4, 0, 3, 128, 16, [3, 60], 128, False, True, False),      # keys and values only
    (1, 70, 3, 3, 64, 16, [5], 16, False, False, False),
])
def test_append(sv, fp8, B, N, Hq, H, D, page, ctx, rot, inter, norm, fused):
    g = torch.Generator().manual_seed(B + 10 * N + D)
    parts = R.make_cache(1, B, max(ctx) + N, page, H, D, fp8, hnd=N % 2 == 1)
    cache = R.on_gpu(sv, parts)
    before = [cache.k.clone(), cache.v.clone()]
    qkv = torch.randn((B, N, Hq + 2 * H, D), generator=g).to(torch.bfloat16)
    q, k, v = qkv.split([Hq, H, H], 2)
    dev = qkv.cuda().split([Hq, H, H], 2)
    if not fused:
        dev = [t.contiguous() for t in dev]
    w = [(torch.rand(D, generator=g) + 0.5).to(torch.bfloat16) if norm else None for _ in range(2)]
    rope = R.rope_table(max(ctx) + N + 5, rot) if rot else None
    c = torch.tensor(ctx, dtype=torch.int32)
    pos = c[:, None] + torch.arange(N)
    given = None
    if B > 1:                                                   # as a tree's depths
        pos = torch.maximum(pos - torch.arange(N) % 3, c[:, None])
        given = pos.to(torch.int32).cuda()
    out = sv.kv_append(cache, dev[0] if Hq else None, dev[1], dev[2], c.cuda(), None if rope is None else rope.cuda(),
                       q_weight=None if w[0] is None else w[0].cuda(), k_weight=None if w[1] is None else w[1].cuda(),
                       eps=1e-5, interleaved=inter, positions=given)
    assert cache.read_error() == 0
    # fp32 steps before the rounding: the norm's D-term sum, its root and two products (D/2 + 8
    # roundings), then one rotation: within (D/2 + 16) u32 of the magnitudes met
    rel = (D / 2 + 16) * R.U_F32
    if Hq:
        y, mag = R.norm_rope(q, w[0], rope, pos, 1e-5, inter)
        assert ((out.cpu().double() - y).abs() <= R.U_BF16 * y.abs() + 1.01 * rel * mag).all()
    y, mag = R.norm_rope(k, w[1], rope, pos, 1e-5, inter)
    touched = torch.zeros(cache.k.shape[:2], dtype=torch.bool)
    for b in range(B):
        t = ctx[b] + torch.arange(N)
        touched[cache.block_table[b].long().cpu()[t // page], t % page] = True
        gk, gv = gather(cache, b, t.cuda())
        for got, want, m in ((gk, y[b], mag[b]), (gv, v[b].double(), v[b].double().abs())):
            if fp8:
                # half a step of a 4-bit significand, or of the smallest step 2^-9 of the scale,
                # with the scale and the quotient in fp32
                sc = want.abs().amax(-1, keepdim=True) / 448
                tol = 2.0 ** -4 * want.abs() + 2.0 ** -10 * sc + 2 * rel * m.amax(-1, keepdim=True)
                assert (got.abs().amax(-1) > 0.99 * want.abs().amax(-1)).all()
            else:
                tol = R.U_BF16 * want.abs() + 1.01 * rel * m
            assert ((got - want).abs() <= tol).all()
    for x, y0 in zip((cache.k, cache.v), before):               # nothing else changed
        same = x.view(torch.uint8 if fp8 else torch.int16) == y0.view(torch.uint8 if fp8 else torch.int16)
        assert same.cpu().flatten(2).all(-1)[~touched].all()


def test_append_quantises_to_the_nearest(sv):
    """Without norm and rotation the stored bytes are the nearest e4m3 of x / scale, to even."""
    D, H = 128, 2
    g = torch.Generator().manual_seed(5)
    k, v = ((torch.randn((1, 9, H, D), generator=g) * torch.pow(10.0, torch.arange(9.0) - 6)[None, :, None, None]).to(torch.bfloat16) for _ in range(2))
    k[0, 3] = 0                                                  # a row of zeros
    k[0, 4, 0, 7] = math.inf
    k[0, 4, 1, 9] = math.nan
    cache = R.on_gpu(sv, R.make_cache(2, 1, 16, 16, H, D, True))
    sv.kv_append(cache, None, k.cuda(), v.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda"))
    pg = int(cache.block_table[0, 0])
    for x, got, sc in ((k, cache.k, cache.k_scale), (v, cache.v, cache.v_scale)):
        a = x[0].float()
        top = torch.where(a.isnan(), torch.zeros(()), a.abs()).amax(-1).clamp_min(1e-20)
        want = top / 448
        assert torch.equal(sc[pg, :9].cpu(), want)
        ref = (a / want[..., None]).clamp(-448, 448).to(R.F8)
        fine = torch.isfinite(a).all(-1)
        assert torch.equal(got[pg, :9].cpu().view(torch.uint8)[fine], ref.view(torch.uint8)[fine])
    back = gather(cache, 0, torch.arange(9, device="cuda"))[0]
    assert (back[3] == 0).all() and not torch.isfinite(back[4, 0, 7]) and torch.isnan(back[4, 1, 9])


def test_append_skips_and_marks(sv):
    """Positions past new_lens are left alone; bad sequences write nothing and give NaN queries."""
    B, N, H, D = 6, 3, 2, 64
    parts = R.make_cache(3, B, 40, 16, H, D)
    parts[2][2, 1] = 10 ** 6
    cache = R.on_gpu(sv, parts)
    k0 = cache.k.clone()
    q, k, v = (torch.ones((B, N, h, D), dtype=torch.bfloat16, device="cuda") for h in (4, H, H))
    ctx = torch.tensor([5, -1, 15, 30, 1000, 7], dtype=torch.int32)
    newl = torch.tensor([2, 3, 3, 0, 3, 3], dtype=torch.int32)
    pos = ctx[:, None] + torch.arange(N)
    pos[5, 1] = 64                                               # past the rope table
    out = torch.full((B, N, 4, D), 7.0, dtype=torch.bfloat16, device="cuda")
    sv.kv_append(cache, q, k, v, ctx.cuda(), R.rope_table(64, D).cuda(), new_lens=newl.cuda(),
                 positions=pos.to(torch.int32).cuda(), out=out)
    assert cache.read_error() == sv.SPEC_DEVERR_CACHE_RANGE
    assert (out[0, 2] == 7).all() and torch.isfinite(out[0, :2]).all() and (out[3] == 7).all()
    assert torch.isnan(out[1]).all() and torch.isnan(out[4]).all()
    assert torch.isfinite(out[2, 0]).all() and torch.isnan(out[2, 1:]).all()
    assert torch.isnan(out[5, 1]).all() and torch.isfinite(out[5, 0]).all()
    wrote = (cache.k.view(torch.int16) != k0.view(torch.int16)).flatten(2).any(-1).sum()
    assert int(wrote) == 2 + 1 + 2


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B,T,H,D,page,dtype", [(1, 1, 1, 64, 16, "bfloat16"), (3, 77, 2, 128, 5, "bfloat16"),
                                               (2, 130, 3, 256, 48, "float32"), (2, 33, 1, 64, 1, "float32")])
def test_read(sv, fp8, B, T, H, D, page, dtype):
    parts = R.make_cache(4, B, T + 9, page, H, D, fp8, hnd=B == 2)
    cache = R.on_gpu(sv, parts)
    dt = getattr(torch, dtype)
    g = torch.Generator().manual_seed(1)
    starts = torch.randint(0, 9, (B,), generator=g).to(torch.int32)
    counts = torch.randint(0, T + 1, (B,), generator=g).to(torch.int32)
    counts[0] = T
    for st, cn in ((None, None), (starts, counts), (starts, None), (None, counts)):
        k, v = sv.kv_read(cache, T, starts=None if st is None else st.cuda(), counts=None if cn is None else cn.cuda(), dtype=dt)
        assert cache.read_error() == 0
        for b in range(B):
            s, n = (0 if st is None else int(st[b])), (T if cn is None else int(cn[b]))
            for x, raw, sc in ((k, parts[0], parts[3]), (v, parts[1], parts[4])):
                t = torch.arange(s, s + n)
                pg = parts[2][b].long()[t // page]
                want = raw.float()[pg, t % page]
                if sc is not None:
                    want = want * sc[pg, t % page][..., None]
                assert torch.equal(x[b, :n].cpu(), want.to(dt))
                assert (x[b, n:] == 0).all()


def test_read_marks_bad_sequences(sv):
    parts = R.make_cache(5, 4, 50, 16, 2, 64)
    parts[2][1, 1] = 999
    cache = R.on_gpu(sv, parts)
    starts = torch.tensor([0, 0, -1, 10 ** 6], dtype=torch.int32).cuda()
    k, v = sv.kv_read(cache, 40, starts=starts)
    assert cache.read_error() == sv.SPEC_DEVERR_CACHE_RANGE and cache.read_error() == 0
    assert torch.isfinite(k[0]).all() and torch.isnan(k[1, 16:32]).all() and torch.isfinite(k[1, :16]).all()
    assert torch.isnan(k[2:]).all() and torch.isnan(v[2:]).all()


def compact_by_hand(parts, layers, ctx, path, acc):
    k, v, table, ks, vs = parts
    page = k.shape[-3]
    out = [None if t is None else t.clone() for t in (k, v, ks, vs)]
    for b in range(len(ctx)):
        if acc[b] <= 0:
            continue
        src = ctx[b] + torch.tensor(path[b][:acc[b]])
        dst = ctx[b] + 1 + torch.arange(acc[b])
        place = lambda t: (table[b].long()[t // page], t % page)  # noqa: E731
        for new, old in zip(out, (k, v, ks, vs)):
            if old is None:
                continue
            bits = lambda x: x.view(torch.uint8) if x.element_size() == 1 else x  # noqa: E731
            for l in range(layers or 1):
                n, o = (bits(new)[l], bits(old)[l]) if layers else (bits(new), bits(old))
                n[place(dst)] = o[place(src)]
    return out


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("layers", [None, 3])
@pytest.mark.parametrize("page,D", [(16, 64), (5, 128), (1, 256)])
def test_compact(sv, fp8, layers, page, D):
    paths = [[1, 2, 3, 4], [3, 4, 5, 6, 7], [], [7], [2, 3, 9], [1, 2, 11], [1, 5, 6, 11], [0], [4, 5, 6, 7, 8, 9, 10, 11]]
    N, B = 12, len(paths)
    acc = [len(p) for p in paths]
    acc[7] = -1                                                  # a sequence that verification marked
    ctx = [0, 3, 10, 15, 16, 31, 7, 5, 20]
    parts = R.make_cache(6, B, max(ctx) + N, page, 2, D, fp8, layers=layers)
    want = compact_by_hand(parts, layers, ctx, paths, acc)
    cache = R.on_gpu(sv, parts)
    path = torch.full((B, N), -1, dtype=torch.int32)
    for b, p in enumerate(paths):
        path[b, :len(p)] = torch.tensor(p, dtype=torch.int32)
    sv.kv_compact(cache, torch.tensor(ctx, dtype=torch.int32).cuda(), path.cuda(), torch.tensor(acc, dtype=torch.int32).cuda())
    assert cache.read_error() == 0
    for got, ref in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), want):
        if ref is not None:
            v = lambda t: t.contiguous().view(torch.uint8)  # noqa: E731
            assert torch.equal(v(got.cpu()), v(ref))


def test_compact_marks_paths_that_are_none(sv):
    parts = R.make_cache(7, 5, 40, 16, 2, 64)
    cache = R.on_gpu(sv, parts)
    before = cache.k.clone()
    path = torch.tensor([[3, 2, -1, -1], [1, 9, -1, -1], [0, 1, -1, -1], [2, 2, -1, -1], [2, 3, -1, -1]], dtype=torch.int32)
    sv.kv_compact(cache, torch.tensor([1, 2, 3, 4, -9], dtype=torch.int32).cuda(), path.cuda(),
                  torch.full((5,), 2, dtype=torch.int32).cuda())
    assert cache.read_error() == sv.SPEC_DEVERR_CACHE_RANGE
    assert torch.equal(cache.k.view(torch.int16), before.view(torch.int16))


def test_streams_and_capture(sv):
    """Appending, attending and reading on a side stream and in a captured graph."""
    B, N, H, D = 2, 4, 2, 128
    parts = R.make_cache(8, B, 200, 16, H, D, True)
    cache = R.on_gpu(sv, parts)
    g = torch.Generator().manual_seed(2)
    q, k, v = (torch.randn((B, N, h, D), generator=g).to(torch.bfloat16).cuda() for h in (8, H, H))
    ctx = torch.tensor([100, 33], dtype=torch.int32).cuda()
    rope = R.rope_table(256, D).cuda()

    def step(stream=None):
        y = sv.kv_append(cache, q, k, v, ctx, rope, stream=stream)
        o = sv.paged_attention(y, cache, ctx, stream=stream)
        return (o, *sv.kv_read(cache, N, starts=ctx, stream=stream))
    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = [step(side) for _ in range(8)]
    torch.cuda.synchronize()
    for r in got:
        assert all(torch.equal(a, b) for a, b in zip(r, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    graph.replay()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(held, want))


def test_refusals(sv):
    B, N, H, D = 2, 3, 2, 64
    cache = R.on_gpu(sv, R.make_cache(9, B, 40, 16, H, D))
    q, k, v = (torch.zeros((B, N, h, D), dtype=torch.bfloat16, device="cuda") for h in (4, H, H))
    ctx = torch.zeros(B, dtype=torch.int32, device="cuda")
    rope = R.rope_table(8, D).cuda()
    ok = dict(cache=cache, q=q, k=k, v=v, context_lens=ctx, rope=rope)

    def bad(err, **kw):
        with pytest.raises(err):
            sv.kv_append(**{**ok, **kw})
    bad(TypeError, q=q.float())
    bad(ValueError, k=k[:, :, :1])
    bad(ValueError, v=v[:1])
    bad(ValueError, rope=rope.double().float().cpu())
    bad(sv.SpecVerifyError, rope=R.rope_table(8, 24).cuda())    # no multiple of 16
    bad(sv.SpecVerifyError, q_weight=torch.ones(D, dtype=torch.bfloat16, device="cuda"), eps=-1.0)
    bad((TypeError, ValueError), context_lens=ctx.long())
    bad(ValueError, context_lens=ctx[:1])
    bad(ValueError, q_weight=torch.ones(D + 1, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(TypeError):
        sv.kv_read(cache, 4, dtype=torch.float16)
    with pytest.raises(ValueError):
        sv.kv_read(cache, 4, counts=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        sv.kv_compact(cache, ctx, torch.zeros((3, 4), dtype=torch.int32, device="cuda"), ctx)
    with pytest.raises(TypeError):
        sv.KVCache(k, v, ctx.long().view(B, 1))
    with pytest.raises(ValueError):
        sv.KVCache(cache.k.transpose(-1, -2), cache.v.transpose(-1, -2), cache.block_table)

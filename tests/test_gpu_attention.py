"""Paged attention of new positions against its 64-bit form (tests/kv_ref.py): chains and
trees, both cache types, head layouts, page sizes, lengths, splits, masked entries that are no
numbers, bad input, streams and captured calls."""
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


def tree(g, B, N):
    p = torch.full((B, N), -1, dtype=torch.int32)
    for n in range(1, N):
        p[:, n] = (torch.rand(B, generator=g) * n).to(torch.int32).clamp(0, n - 1)
    return p


def case(seed, B, N, Hq, H, D, page, ctx, fp8=False, hnd=False, is_tree=False, newl=None, qscale=1.5):
    g = torch.Generator().manual_seed(seed + 1)
    parts = R.make_cache(seed, B, max(ctx) + N, page, H, D, fp8, hnd)
    q = (torch.randn((B, N, Hq, D), generator=g) * qscale).to(torch.bfloat16)
    par = tree(g, B, N) if is_tree else None
    c = torch.tensor(ctx, dtype=torch.int32)
    nb = torch.full((B,), N, dtype=torch.int32) if newl is None else torch.tensor(newl, dtype=torch.int32)
    return parts, q, par, c, nb


def check(sv, parts, q, par, c, nb, scale=None, **kw):
    cache = R.on_gpu(sv, parts)
    out, lse = sv.paged_attention(q.cuda(), cache, c.cuda(), parents=None if par is None else par.cuda(),
                                  new_lens=nb.cuda(), scale=scale, lse=True, **kw)
    o, l, to, tl = R.attention(q, *parts, c, nb, par, scale)
    assert cache.read_error() == 0
    out, lse = out.cpu().double(), lse.cpu().double()
    assert torch.isfinite(out).all()
    worst = ((out - o).abs() / to.clamp_min(1e-30)).max()
    assert ((out - o).abs() <= to).all(), f"out off by {worst} of its tolerance"
    assert torch.equal(torch.isinf(lse), torch.isinf(l))
    fin = torch.isfinite(l)
    assert ((lse - l).abs()[fin] <= tl[fin]).all(), "lse"
    return out


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B,N,Hq,H,D,page,ctx", [
    (1, 1, 1, 1, 64, 16, [0]),                       # one position that sees itself alone
    (1, 1, 32, 8, 128, 16, [777]),
    (3, 1, 8, 1, 128, 1, [0, 1, 130]),               # pages of one position
    (2, 8, 8, 2, 128, 64, [63, 64]),                 # 32 rows; a page's end at, and inside, the new positions
    (2, 5, 10, 2, 128, 5, [7, 201]),                 # odd everything
    (4, 3, 4, 4, 64, 48, [15, 16, 17, 333]),
    (1, 17, 12, 12, 64, 16, [99]),
    (2, 9, 16, 2, 128, 16, [40, 3]),                 # 72 rows: several row blocks
    (1, 2, 6, 2, 256, 16, [500]),
    (2, 7, 14, 2, 256, 32, [31, 65]),
    (1, 3, 64, 1, 128, 16, [70]),                    # all query heads on one cached head
    (1, 33, 2, 1, 64, 16, [20]),
])
def test_chains(sv, fp8, B, N, Hq, H, D, page, ctx):
    check(sv, *case(B * 100 + N, B, N, Hq, H, D, page, ctx, fp8, hnd=N % 2 == 0))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B,N,Hq,H,D,ctx", [(2, 2, 4, 2, 64, [0, 5]), (2, 36, 8, 2, 128, [100, 17]),
                                           (1, 64, 4, 1, 128, [63]), (1, 64, 2, 2, 256, [1]),
                                           (3, 11, 8, 8, 64, [0, 250, 31])])
def test_trees(sv, fp8, B, N, Hq, H, D, ctx):
    check(sv, *case(N, B, N, Hq, H, D, 16, ctx, fp8, is_tree=True))


def test_tree_shaped_as_a_chain_is_a_chain(sv):
    parts, q, _, c, nb = case(3, 2, 8, 8, 2, 128, 16, [100, 37])
    cache = R.on_gpu(sv, parts)
    par = (torch.arange(8, dtype=torch.int32) - 1).repeat(2, 1)
    a = sv.paged_attention(q.cuda(), cache, c.cuda())
    b = sv.paged_attention(q.cuda(), cache, c.cuda(), parents=par.cuda())
    assert torch.equal(a, b)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("N", [2, 5, 12, 36])                     # 8, 20, 48 and 144 rows of a cached head
def test_long_context_is_split_and_joined(sv, fp8, N):
    """One sequence over every CTA, ragged beside short ones, and the same bits every time."""
    args = case(5, 3, N, 8, 2, 128, 16, [9001, 3, 1500], fp8)
    check(sv, *args)
    parts, q, _, c, nb = args
    cache = R.on_gpu(sv, parts)
    runs = [sv.paged_attention(q.cuda(), cache, c.cuda()) for _ in range(5)]
    assert all(torch.equal(runs[0], r) for r in runs)


def test_longest_chain(sv):
    check(sv, *case(8, 1, 257, 1, 1, 64, 16, [40]))


@pytest.mark.parametrize("is_tree", [False, True])
def test_ragged_new_lengths_and_empty_rows(sv, is_tree):
    """Rows past a sequence's new positions are zero with lse -inf; a sequence may have none."""
    args = case(9, 5, 6, 8, 2, 128, 16, [10, 0, 77, 0, 200], is_tree=is_tree, newl=[6, 1, 0, 0, 3])
    out = check(sv, *args)
    assert (out[2] == 0).all() and (out[4, 3:] == 0).all() and (out[4, :3] != 0).any()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_masked_entries_may_hold_anything(sv, value, fp8):
    """A branch's keys, values and scales that are no numbers reach only the rows that see it."""
    if fp8 and value != math.nan:
        value = math.nan
    parts, q, _, c, nb = case(11, 1, 20, 4, 2, 128, 16, [30], fp8)
    par = torch.tensor([[-1, 0, 1, 2, 3] + [0] * 15], dtype=torch.int32)    # node 7 is a leaf
    k, v, table, ks, vs = parts
    pos = 30 + 7
    at = (int(table[0, pos // 16]), pos % 16)
    clean = R.on_gpu(sv, parts)
    want, wl = sv.paged_attention(q.cuda(), clean, c.cuda(), parents=par.cuda(), lse=True)
    for name in (k, v):
        x = name.float()
        x[at[0], at[1], :, 5:9] = value
        name.copy_(x.to(name.dtype))
    cache = R.on_gpu(sv, parts)
    got, gl = sv.paged_attention(q.cuda(), cache, c.cuda(), parents=par.cuda(), lse=True)
    others = [n for n in range(20) if n != 7]
    assert torch.equal(got[:, others], want[:, others]) and torch.equal(gl[:, others], wl[:, others])
    assert not torch.isfinite(got[:, 7]).all()
    # a value alone, seen by its own row: no number where it is none, the rest as before
    parts2, *_ = case(11, 1, 20, 4, 2, 128, 16, [30], fp8)
    x = parts2[1].float()
    x[at[0], at[1], :, 5] = value
    parts2[1].copy_(x.to(parts2[1].dtype))
    got = sv.paged_attention(q.cuda(), R.on_gpu(sv, parts2), c.cuda(), parents=par.cuda())
    assert torch.equal(got[:, others], want[:, others])
    bad = ~torch.isfinite(got[:, 7].float())
    assert bad[..., 5].all() and not bad[..., 6:].any() and not bad[..., :5].any()
    diff = (got[:, 7].float() - want[:, 7].float()).abs()
    ok = ~bad
    assert (diff[ok] <= 2.0 ** -6 * want[:, 7].float().abs()[ok] + 2.0 ** -6).all()


def test_scores_of_any_size(sv):
    """Large scores (a softmax of one entry), equal scores, and a negative scale."""
    for qscale, scale in ((60.0, None), (0.0, None), (1.0, -0.2), (1.0, 0.0)):
        check(sv, *case(13, 2, 4, 8, 2, 128, 16, [100, 259], qscale=qscale), scale=scale)
        check(sv, *case(13, 2, 4, 8, 2, 128, 16, [100, 259], fp8=True, qscale=qscale), scale=scale)


def test_value_scales_far_apart(sv):
    """An 8-bit cache whose positions' value scales span many powers of two, zeros among
    the rows."""
    parts, q, par, c, nb = case(14, 1, 4, 8, 2, 128, 16, [300], fp8=True)
    g = torch.Generator().manual_seed(3)
    parts[4].copy_(parts[4] * torch.pow(2.0, torch.randint(-40, 10, parts[4].shape, generator=g).float()))
    check(sv, parts, q, par, c, nb)


def test_strided_queries_and_joint_pool(sv):
    """Queries sliced from a fused projection; keys beside values in one tensor."""
    B, N, Hq, H, D, page = 2, 4, 8, 2, 128, 16
    parts, q, par, c, nb = case(15, B, N, Hq, H, D, page, [50, 90])
    k, v, table, _, _ = parts
    pool = torch.stack([k, v], 1).cuda()                       # [pages, 2, page, H, D]
    cache = sv.KVCache(pool[:, 0], pool[:, 1], table.cuda())
    fused = torch.randn((B, N, Hq + 2 * H, D)).to(torch.bfloat16)
    fused[:, :, :Hq] = q
    out = sv.paged_attention(fused.cuda()[:, :, :Hq], cache, c.cuda())
    o, _, to, _ = R.attention(q, *parts, c, nb)
    assert ((out.cpu().double() - o).abs() <= to).all()


def test_offsets_past_32_bits(sv):
    """Pages whose elements lie beyond 2^32 of the cache's first."""
    page, H, D, N = 64, 8, 128, 2
    pages = (1 << 32) // (page * H * D) + 40
    k = torch.empty((pages, page, H, D), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    parts, q, par, c, nb = case(16, 1, N, 8, H, D, page, [150])
    high = torch.tensor([[pages - 1, pages - 30, 3, pages - 2, -1]], dtype=torch.int32)
    for i in range(3):
        k[int(high[0, i])] = parts[0][int(parts[2][0, i])].cuda()
        v[int(high[0, i])] = parts[1][int(parts[2][0, i])].cuda()
    out = sv.paged_attention(q.cuda(), sv.KVCache(k, v, high.cuda()), c.cuda())
    o, _, to, _ = R.attention(q, *parts, c, nb)
    assert ((out.cpu().double() - o).abs() <= to).all()


def test_bad_sequences_are_marked_and_the_others_hold(sv):
    parts, q, _, c, nb = case(17, 6, 4, 8, 2, 128, 16, [40, 100, 60, 20, 30, 1000])
    good = R.on_gpu(sv, parts)
    want = sv.paged_attention(q.cuda(), good, c.cuda())
    table = parts[2].clone()
    table[1, 2] = 1 << 20                                       # a page that is none
    table[2, 0] = -5
    c2, n2 = c.clone(), nb.clone()
    c2[3] = -1
    n2[4] = 5                                                   # more than the call brings
    c2[5] = table.shape[1] * 16 - 3                             # runs past the table
    cache = R.on_gpu(sv, (parts[0], parts[1], table, None, None))
    got, lse = sv.paged_attention(q.cuda(), cache, c2.cuda(), new_lens=n2.cuda(), lse=True)
    assert cache.read_error() == sv.SPEC_DEVERR_CACHE_RANGE
    assert torch.equal(got[0], want[0])
    assert torch.isnan(got[1:]).all() and torch.isnan(lse[1:]).all()
    assert torch.equal(sv.paged_attention(q.cuda(), good, c.cuda()), want)


def test_malformed_trees(sv):
    parts, q, _, c, nb = case(18, 3, 4, 4, 2, 64, 16, [20, 30, 40])
    par = torch.tensor([[-1, 0, 1, 1], [0, 0, 1, 1], [-1, 0, 2, 1]], dtype=torch.int32)
    cache = R.on_gpu(sv, parts)
    out = sv.paged_attention(q.cuda(), cache, c.cuda(), parents=par.cuda())
    assert cache.read_error() == sv.SPEC_DEVERR_TREE_PARENT
    assert torch.isfinite(out[0]).all() and torch.isnan(out[1:]).all()


def test_one_workspace_for_calls_of_every_size(sv):
    """Calls of different sizes in turn through one workspace, nothing waiting between them."""
    ws = torch.zeros(sv.load_library().spec_attention_workspace_size(8, 64, 32, 2, 128), dtype=torch.uint8, device="cuda")
    sizes = [(20, 1, 8, 32, 8, 128, [2000], False), (21, 3, 36, 8, 2, 128, [700, 30, 1500], True),
             (22, 2, 3, 4, 4, 64, [4000, 100], False), (23, 1, 64, 2, 1, 128, [900], True)]
    held = []
    for seed, B, N, Hq, H, D, ctx, tr in sizes:
        parts, q, par, c, nb = case(seed, B, N, Hq, H, D, 16, ctx, is_tree=tr)
        cache = R.on_gpu(sv, parts)
        kw = dict(parents=None if par is None else par.cuda())
        held.append((q.cuda(), cache, c.cuda(), kw, sv.paged_attention(q.cuda(), cache, c.cuda(), **kw)))
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        got.append([sv.paged_attention(q, cache, c, workspace=ws, **kw) for q, cache, c, kw, _ in held])
    for row in got:
        for x, (_, _, _, _, want) in zip(row, held):
            assert torch.equal(x, want)


def test_on_another_stream(sv):
    parts, q, par, c, nb = case(24, 2, 4, 8, 2, 128, 16, [1000, 5000])
    cache, qd, cd = R.on_gpu(sv, parts), q.cuda(), c.cuda()
    want = sv.paged_attention(qd, cache, cd)
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(3)]
    outs = [sv.paged_attention(qd, cache, cd, stream=s) for _ in range(20) for s in side]
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o in outs)


def test_captured_call_follows_its_lengths(sv):
    parts, q, par, c, nb = case(25, 2, 2, 8, 2, 128, 16, [3000, 40])
    cache, qd, cd = R.on_gpu(sv, parts), q.cuda(), c.cuda()
    out = torch.empty_like(qd)
    sv.paged_attention(qd, cache, cd, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sv.paged_attention(qd, cache, cd, out=out)
    for lens in ([3000, 40], [7, 2900], [0, 0], [1234, 999]):
        cd.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        got = out.clone()
        assert torch.equal(got, sv.paged_attention(qd, cache, cd))


def test_refusals(sv):
    parts, q, par, c, nb = case(26, 2, 4, 8, 2, 128, 16, [10, 20])
    cache, qd, cd = R.on_gpu(sv, parts), q.cuda(), c.cuda()
    with pytest.raises(TypeError):
        sv.paged_attention(qd.float(), cache, cd)
    with pytest.raises(ValueError):
        sv.paged_attention(qd[:, :, :, :64], cache, cd)
    with pytest.raises(ValueError):
        sv.paged_attention(qd[:, :, :7].contiguous(), cache, cd)
    with pytest.raises(ValueError):
        sv.paged_attention(qd.transpose(1, 2).contiguous().transpose(1, 2), cache, cd)
    with pytest.raises((TypeError, ValueError)):
        sv.paged_attention(qd, cache, cd.long())
    with pytest.raises(ValueError):
        sv.paged_attention(qd, cache, cd[:1])
    with pytest.raises(sv.SpecVerifyError):
        sv.paged_attention(qd, cache, cd, scale=math.inf)
    with pytest.raises(sv.SpecVerifyError):
        sv.paged_attention(qd, cache, cd, workspace=torch.zeros(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        sv.KVCache(cache.k, cache.v[:, :, :1], cache.block_table)
    with pytest.raises(ValueError):
        sv.KVCache(cache.k, cache.v, cache.block_table, torch.zeros(3, device="cuda"))


@pytest.mark.parametrize("fp8", [False, True])
def test_waits_that_run_out_report_and_return(sv, fp8):
    """With the kernels' bounded waits set to give up at once: the error word says so, the rows
    are NaN, and later calls through the same workspace are right again."""
    args = case(27, 2, 10, 8, 2, 128, 16, [700, 3000], fp8)       # 40 rows: the kernel that has waits
    parts, q, par, c, nb = args
    cache = R.on_gpu(sv, parts)
    want = sv.paged_attention(q.cuda(), cache, c.cuda())
    torch.cuda.synchronize()
    sv.spec_verify_set_wait_limit(0)
    try:
        out = sv.paged_attention(q.cuda(), cache, c.cuda())
        torch.cuda.synchronize()
    finally:
        sv.spec_verify_set_wait_limit(sv.spec_verify_default_wait_limit())
    assert cache.read_error() & sv.SPEC_DEVERR_TIMEOUT
    assert torch.isnan(out).all()
    assert torch.equal(sv.paged_attention(q.cuda(), cache, c.cuda()), want)
    assert cache.read_error() == 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page", [8, 16, 64, 128, 256, 48])
@pytest.mark.parametrize("Hq", [16, 64, 160])                   # 6, 24 and 60 rows of a cached head
def test_long_shares(sv, fp8, page, Hq):
    """Shares of many tiles, old positions and new ones in turn, against the rows one by one: every
    sequence's answer is that of the sequence alone."""
    g = torch.Generator().manual_seed(page)
    B, N, H, D = 40, 3, 8, 128
    ctx = torch.randint(0, 3000, (B,), generator=g).tolist()
    cache = sv.KVCache(*R.make_cache_on_gpu(28, B, max(ctx) + N, page, H, D, fp8))
    qd = (torch.randn((B, N, Hq, D), generator=g) * 1.5).to(torch.bfloat16).cuda()
    cd = torch.tensor(ctx, dtype=torch.int32).cuda()
    whole = [sv.paged_attention(qd, cache, cd) for _ in range(4)]
    assert all(torch.equal(w, whole[0]) for w in whole)
    assert cache.read_error() == 0
    for b in range(0, B, 7):
        one = sv.KVCache(cache.k, cache.v, cache.block_table[b:b + 1].contiguous(), cache.k_scale, cache.v_scale)
        alone = sv.paged_attention(qd[b:b + 1].contiguous(), one, cd[b:b + 1].contiguous())
        # the split differs, so sums come in another order and references differ: P and the
        # result are each rounded anew (two unit roundoffs of the values' magnitude, at most 4.5)
        assert (alone.float() - whole[0][b:b + 1].float()).abs().max() <= 4.5 * 2 * R.U_BF16


@pytest.mark.parametrize("N", [2, 12])
def test_scale_of_zero(sv, N):
    """An 8-bit position whose value scale is zero has a value of zero and keeps its weight."""
    parts, q, par, c, nb = case(29, 1, N, 8, 2, 128, 16, [200], fp8=True)
    parts[4].view(-1)[::3] = 0.0
    check(sv, parts, q, par, c, nb)


@pytest.mark.parametrize("N,G", [(6, 4), (7, 5), (16, 1), (33, 1), (5, 7), (64, 2), (1, 40)])
@pytest.mark.parametrize("fp8", [False, True])
def test_rows_around_the_kernels_bounds(sv, fp8, N, G):
    """Row counts on both sides of 16, 32, 64 and 144, in a table with room for long contexts."""
    parts = R.make_cache(30 + N, 2, 300, 16, 2, 128, fp8, max_pages=200)
    g = torch.Generator().manual_seed(N)
    q = (torch.randn((2, N, 2 * G, 128), generator=g) * 1.5).to(torch.bfloat16)
    check(sv, parts, q, None, torch.tensor([200, 77], dtype=torch.int32), torch.full((2,), N, dtype=torch.int32))


@pytest.mark.parametrize("N,Hq,H,D,ctx", [(1, 32, 8, 128, [2000]), (9, 32, 8, 128, [3000, 40, 1]), (16, 8, 1, 64, [1300, 0]),
                                          (13, 4, 1, 128, [4749]), (12, 8, 1, 256, [2000, 1999])])
def test_workspace_of_any_contents(sv, N, Hq, H, D, ctx):
    """What lies in the workspace before a call does not matter: results are those of a clear one,
    and right (the many parts of one long unit are joined by several warps a row)."""
    parts, q, par, c, nb = case(31, len(ctx), N, Hq, H, D, 16, ctx)
    cache = R.on_gpu(sv, parts)
    n = sv.load_library().spec_attention_workspace_size(len(ctx), N, Hq, H, D)
    got = [sv.paged_attention(q.cuda(), cache, c.cuda(), lse=True, workspace=torch.full((n,), fill, dtype=torch.uint8, device="cuda"))
           for fill in (0, 255, 1)]
    for o, l in got[1:]:
        assert torch.equal(o, got[0][0]) and torch.equal(l, got[0][1])
    check(sv, parts, q, par, c, nb)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("layout", ["heads outermost", "keys beside values", "odd page step", "pages reversed in steps of two"])
@pytest.mark.parametrize("page", [8, 16, 64, 256])
def test_cache_layouts(sv, fp8, layout, page):
    """Layers whose pages lie in other ways than one after another, whichever way the kernel brings
    them: results are those of the plain layout."""
    B, N, Hq, H, D, ctx = 2, 9, 8, 2, 128, [2700, 300]
    parts, q, par, c, nb = case(33, B, N, Hq, H, D, page, ctx, fp8=fp8)
    k, v, table, ks, vs = parts
    want = sv.paged_attention(q.cuda(), R.on_gpu(sv, parts), c.cuda(), lse=True)
    P = k.shape[0]

    def lay(x):
        x = x.cuda()
        if layout == "heads outermost":
            return x.permute(2, 0, 1, 3).contiguous().permute(1, 2, 0, 3)
        if layout == "odd page step":                      # 16 bytes between pages
            big = torch.zeros(P, page * H * D + 16 // x.element_size(), device="cuda", dtype=torch.uint8 if fp8 else x.dtype)
            y = big.view(x.dtype)[:, :page * H * D].view(P, page, H, D)
        elif layout == "keys beside values":
            y = torch.zeros(P, page, H, 2, D, device="cuda", dtype=torch.uint8 if fp8 else x.dtype).view(x.dtype)[:, :, :, 1]
        else:
            y = torch.zeros(2 * P, page, H, D, device="cuda", dtype=torch.uint8 if fp8 else x.dtype).view(x.dtype)[::2]
        y.copy_(x)
        return y
    cache = sv.KVCache(lay(k), lay(v), table.cuda(), None if ks is None else ks.cuda(), None if vs is None else vs.cuda())
    got = sv.paged_attention(q.cuda(), cache, c.cuda(), lse=True)
    assert cache.read_error() == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("is_tree", [False, True])
@pytest.mark.parametrize("Hq,H,ctx", [(8, 2, [60 + 7 * b for b in range(40)]), (6, 1, [40000]), (8, 4, [b % 3 for b in range(30)])])
def test_wide_heads_many_rows(sv, is_tree, Hq, H, ctx):
    """Heads of 256, more rows than a matrix tile holds, many blocks of them or many tiles."""
    check(sv, *case(35, len(ctx), 11, Hq, H, 256, 16, ctx, is_tree=is_tree,
                    newl=[11 - b % 4 for b in range(len(ctx))]))


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("H", [2, 8])
def test_wide_heads_masked_values(sv, value, H):
    """The same with branches' values that are no numbers, several in a slice: only the rows that see
    them have none, where they have none."""
    B = 24
    parts, q, _, c, nb = case(36, B, 12, 4 * H, H, 256, 16, [21 + b for b in range(B)])
    par = torch.tensor([[-1, 0, 1, 2] + [0] * 8] * B, dtype=torch.int32)    # nodes 4 to 11 are leaves
    want = sv.paged_attention(q.cuda(), R.on_gpu(sv, parts), c.cuda(), parents=par.cuda())
    table = parts[2]
    for b in range(B):
        for n in (5, 6, 9):
            pos = 21 + b + n
            parts[1][int(table[b, pos // 16]), pos % 16, :, n::64] = value
    got = sv.paged_attention(q.cuda(), R.on_gpu(sv, parts), c.cuda(), parents=par.cuda())
    for n in range(12):
        bad = torch.zeros(256, dtype=torch.bool, device="cuda")
        if n in (5, 6, 9):
            bad[n::64] = True
        assert not torch.isfinite(got[:, n][..., bad].float()).any()
        assert torch.isfinite(got[:, n][..., ~bad].float()).all()
        if n not in (5, 6, 9):
            assert torch.equal(got[:, n], want[:, n])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("B,N,Hq,H,D,longest", [(3, 1, 8, 2, 128, 200), (3, 1, 8, 2, 128, 300), (12, 11, 32, 8, 128, 420),
                                                (2, 11, 32, 8, 128, 420), (60, 9, 16, 8, 128, 700), (5, 9, 16, 8, 128, 700),
                                                (50, 5, 32, 8, 64, 500), (70, 2, 16, 8, 256, 240)])
def test_units_whole_and_split(sv, fp8, B, N, Hq, H, D, longest):
    """Short contexts on both sides of the bounds up to which a head's positions stay together, the
    empty one among them, more units than fit at once and fewer."""
    g = torch.Generator().manual_seed(longest + B)
    ctx = torch.randint(0, longest, (B,), generator=g).tolist()
    ctx[0], ctx[-1] = longest - N, 0
    check(sv, *case(41, B, N, Hq, H, D, 16, ctx, fp8=fp8, newl=[N - b % 2 for b in range(B)]))

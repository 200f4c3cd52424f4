"""Paged attention where scores, probabilities and scales lie far apart, for every row count that
picks another kernel or another form of one, against the 64-bit form (tests/kv_ref.py): one
score far above a long context, scores of any size, value scales many powers of two apart, and
masked positions whose scales are no numbers."""
import math

import pytest

torch = pytest.importorskip("torch")
import kv_ref as R  # noqa: E402

pytestmark = pytest.mark.gpu

ROWS = [(4, 4), (5, 4), (12, 4), (16, 4), (36, 4)]            # 16, 20, 48, 64 and 144 rows of a cached head


@pytest.fixture(scope="module")
def sv():
    import __graft_entry__
    __graft_entry__.build()
    import speculative_decoding_verification_59_gb300 as m
    return m


def quantise(x):
    """E4M3 with one scale a row, as the append writes it."""
    sc = x.abs().amax(-1).clamp_min(1e-20) / 448
    return (x / sc[..., None]).to(R.F8), sc


def steps(q, k, v, ks, vs, c, nb, table, parents=None, scale=None):
    """What the smallest step of a probability can leave out, [B, N, Hq, D].

    A probability of an 8-bit cache is held with its position's value scale, in steps of
    2^-23 of the largest such product of its row at most (2^-24 either way)."""
    if ks is None:
        return 0.0
    B, N, Hq, D = q.shape
    G = Hq // k.shape[-2]
    out = torch.zeros((B, N, Hq, D), dtype=torch.float64)
    for b in range(B):
        n, cb = int(nb[b]), int(c[b])
        K = R.rows(k, ks, table, b, cb + n)
        V8 = R.rows(v, None, table, b, cb + n)                 # as held, without their scales
        t = torch.arange(cb + n)
        page = v.shape[-3]
        S = vs[table[b].long()[t // page], t % page].double()
        for h in range(Hq):
            for i in range(n):
                x = (K[:, h // G] @ q[b, i, h].double()) * (D ** -0.5 if scale is None else scale)
                sees = torch.ones(cb + n, dtype=torch.bool)
                sees[cb:] = torch.arange(n) <= i if parents is None else R.ancestors(parents[b, :n])[i]
                p = torch.softmax(x.masked_fill(~sees, -math.inf), 0)
                out[b, i, h] = 2.0 ** -24 * (p * S[:, h // G]).max() * V8[sees, h // G].abs().sum(0)
    return out


def check(sv, parts, q, par, c, nb, scale=None):
    cache = R.on_gpu(sv, parts)
    out, lse = sv.paged_attention(q.cuda(), cache, c.cuda(), parents=None if par is None else par.cuda(),
                                  new_lens=nb.cuda(), scale=scale, lse=True)
    k, v, table, ks, vs = parts
    o, l, to, tl = R.attention(q, *parts, c, nb, par, scale)
    to = to + steps(q, k, v, ks, vs, c, nb, table, par, scale)
    assert cache.read_error() == 0
    out, lse = out.cpu().double(), lse.cpu().double()
    assert torch.isfinite(out).all()
    worst = ((out - o).abs() / to.clamp_min(1e-30)).max()
    assert ((out - o).abs() <= to).all(), f"out off by {worst} of its tolerance"
    assert ((lse - l).abs() <= tl).all(), "lse"


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("N,G,ctx,bits", [(*r, 8192, 18) for r in ROWS] + [(5, 4, 13000, 15), (12, 4, 5000, 20), (4, 4, 13000, 20)])
def test_one_score_far_above_a_long_context(sv, fp8, N, G, ctx, bits):
    """The first position's score lies `bits` powers of two above thousands of others, whose values
    agree on a mean: together they carry a few per cent of the weight, each next to nothing."""
    D, page = 128, 16
    g = torch.Generator().manual_seed(bits + N)
    T = ctx + N
    pages = -(-T // page)
    table = torch.randperm(pages, generator=g)[None].to(torch.int32)
    k = torch.randn((T, 1, D), generator=g) * 0.3
    v = torch.randn((T, 1, D), generator=g) * 0.2 + 1.0
    q = torch.randn((1, N, G, D), generator=g) * 0.5
    q[..., 0] = 8.0
    k[:, :, 0] = 0.0
    k[0, :, 0] = bits * math.log(2) / (8.0 * D ** -0.5)
    v[0] = torch.randn((1, D), generator=g)

    def paged(x):
        y = torch.zeros((pages, page, *x.shape[1:]), dtype=torch.float32)
        t = torch.arange(T)
        y[table[0].long()[t // page], t % page] = x
        return y
    kp, vp = paged(k), paged(v)
    if fp8:
        (kp, ks), (vp, vs) = quantise(kp), quantise(vp)
    else:
        kp, vp, ks, vs = kp.to(torch.bfloat16), vp.to(torch.bfloat16), None, None
    check(sv, (kp, vp, table, ks, vs), q.to(torch.bfloat16), None, torch.tensor([ctx], dtype=torch.int32),
          torch.tensor([N], dtype=torch.int32))


def case(seed, N, G, ctx, fp8, qscale=1.5, is_tree=False):
    """Two sequences, two cached heads, in a table with room for long contexts."""
    parts = R.make_cache(seed, 2, max(ctx) + N, 16, 2, 128, fp8, max_pages=200)
    g = torch.Generator().manual_seed(seed + 1)
    q = (torch.randn((2, N, 2 * G, 128), generator=g) * qscale).to(torch.bfloat16)
    par = None
    if is_tree:
        par = torch.full((2, N), -1, dtype=torch.int32)
        for n in range(1, N):
            par[:, n] = (torch.rand(2, generator=g) * n).to(torch.int32).clamp(0, n - 1)
    return parts, q, par, torch.tensor(ctx, dtype=torch.int32), torch.full((2,), N, dtype=torch.int32)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("N,G", ROWS)
@pytest.mark.parametrize("qscale,scale", [(60.0, None), (0.0, None), (1.0, -0.2), (1.0, 0.0)])
def test_scores_of_any_size(sv, fp8, N, G, qscale, scale):
    """Large scores (a softmax of one entry), equal scores, and a negative scale."""
    check(sv, *case(13, N, G, [100, 459], fp8, qscale, is_tree=N == 12), scale=scale)


@pytest.mark.parametrize("N,G", ROWS)
def test_rising_scores(sv, N, G):
    """Every tile's scores lie above those of the tile before, by more and by less than what moves a
    row's reference."""
    for step in (1.0, 3.0, 12.0):
        for fp8 in (False, True):
            parts, q, par, c, nb = case(15, N, G, [1000, 640], fp8)
            k, v, table, ks, vs = parts
            q = q.clone()
            q[..., 0] = 4.0
            t = torch.arange(1000 + N)
            for b in range(2):
                tb = t[t < int(c[b]) + N]
                at = (table[b].long()[tb // 16], tb % 16)
                x = R.rows(k, ks, table, b, len(tb)).float()
                x[..., 0] = (step * math.log(2) * (tb // 128) / (4.0 * 128 ** -0.5)).float()[:, None]
                if fp8:
                    y, ks[at] = quantise(x)
                    k.view(torch.uint8)[at] = y.view(torch.uint8)
                else:
                    k[at] = x.to(torch.bfloat16)
            check(sv, parts, q, par, c, nb)


@pytest.mark.parametrize("N,G", ROWS)
def test_value_scales_far_apart(sv, N, G):
    """An 8-bit cache whose positions' value scales span many powers of two."""
    parts, q, par, c, nb = case(14, N, G, [300, 77], True)
    g = torch.Generator().manual_seed(3)
    parts[4].copy_(parts[4] * torch.pow(2.0, torch.randint(-40, 10, parts[4].shape, generator=g).float()))
    check(sv, parts, q, par, c, nb)


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("N,G", [(8, 2), (16, 2), (20, 2), (36, 4)])
def test_masked_scales_may_be_anything(sv, value, N, G):
    """A branch's scales that are no numbers reach only the rows that see it."""
    parts, q, _, c, nb = case(11, N, G, [30, 190], True)
    table = parts[2]
    par = torch.tensor([[-1, 0, 1, 2, 3] + [0] * (N - 5)] * 2, dtype=torch.int32)    # node 7 is a leaf
    want, wl = sv.paged_attention(q.cuda(), R.on_gpu(sv, parts), c.cuda(), parents=par.cuda(), lse=True)
    for which in ((3,), (4,), (3, 4)):
        changed = [t.clone() for t in parts]
        for b in range(2):
            pos = int(c[b]) + 7
            for i in which:
                changed[i][int(table[b, pos // 16]), pos % 16] = value
        got, gl = sv.paged_attention(q.cuda(), R.on_gpu(sv, changed), c.cuda(), parents=par.cuda(), lse=True)
        others = [n for n in range(N) if n != 7]
        assert torch.equal(got[:, others], want[:, others]) and torch.equal(gl[:, others], wl[:, others])
        if value != value or 4 in which:                       # (a key scale of infinity may mask the position)
            assert not torch.isfinite(got[:, 7]).any()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("N,G", ROWS)
@pytest.mark.parametrize("ctx,bits", [(6000, 18), (2500, 16)])
def test_one_score_far_above_in_long_shares(sv, fp8, N, G, ctx, bits):
    """The same where a row meets the far score and most others in one running sum: 128 or 192
    sequences and heads, fewer and more than there are multiprocessors, over the same pages with
    the same queries."""
    D, page, B, H = 128, 16, 16 if ctx > 3000 else 24, 8
    g = torch.Generator().manual_seed(bits + N)
    T = ctx + N
    pages = -(-T // page)
    k = torch.randn((pages * page, 1, D), generator=g) * 0.3
    v = torch.randn((pages * page, 1, D), generator=g) * 0.2 + 1.0
    q = torch.randn((1, N, G, D), generator=g) * 0.5
    q[..., 0] = 8.0
    k[:, :, 0] = 0.0
    k[3, :, 0] = bits * math.log(2) / (8.0 * D ** -0.5)
    v[3] = torch.randn((1, D), generator=g)
    k, v, q = k.view(pages, page, 1, D), v.view(pages, page, 1, D), q.to(torch.bfloat16)
    if fp8:
        (k, ks), (v, vs) = quantise(k), quantise(v)
    else:
        k, v, ks, vs = k.to(torch.bfloat16), v.to(torch.bfloat16), None, None
    table = torch.arange(pages, dtype=torch.int32)[None]
    c, nb = torch.tensor([ctx], dtype=torch.int32), torch.tensor([N], dtype=torch.int32)
    o, l, to, tl = R.attention(q, k, v, table, ks, vs, c, nb)
    to = to + steps(q, k, v, ks, vs, c, nb, table)

    def wide(x):
        return None if x is None else x.float().expand(pages, page, H, *x.shape[3:]).to(x.dtype).cuda()
    cache = sv.KVCache(wide(k), wide(v), table.repeat(B, 1).cuda(), *(() if ks is None else (wide(ks), wide(vs))))
    many = q[:, :, None].expand(B, N, H, G, D).reshape(B, N, H * G, D).cuda()
    out, lse = sv.paged_attention(many, cache, c.repeat(B).cuda(), lse=True)
    assert cache.read_error() == 0
    out, lse = out.cpu().double().view(B, N, H, G, D), lse.cpu().double().view(B, N, H, G)
    for h in range(H):
        worst = ((out[:, :, h] - o).abs() / to).max()
        assert worst <= 1, f"out off by {worst} of its tolerance"
        assert ((lse[:, :, h] - l).abs() <= tl).all()

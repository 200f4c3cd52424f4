"""The target model's dense side against its plain forms in 64 bits."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import linear_ref as R  # noqa: E402


@pytest.fixture(scope="module")
def sv():
    import __graft_entry__
    __graft_entry__.build()
    import speculative_decoding_verification_59_gb300 as m
    return m


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


# ---- residual and norm -----------------------------------------------------------------
@pytest.mark.parametrize("rows,dim", [(1, 16), (3, 64), (5, 128), (2, 144), (33, 1008), (7, 4096), (300, 4096), (2, 8192), (3, 16384),
                                      (2, 16400), (3, 40000)])
@pytest.mark.parametrize("xt,rt", [("bfloat16", "bfloat16"), ("bfloat16", "float32"), ("float32", "bfloat16"), ("float32", None)])
@pytest.mark.parametrize("out", ["bf16", "f32", "e4m3"])
def test_add_norm(sv, rows, dim, xt, rt, out):
    g = gen(rows * dim)
    x = torch.randn((rows, dim), generator=g, device="cuda").to(getattr(torch, xt))
    r = None if rt is None else (3 * torch.randn((rows, dim), generator=g, device="cuda")).to(getattr(torch, rt))
    w = None if dim == 1008 else (torch.rand(dim, generator=g, device="cuda") + 0.5).to(torch.bfloat16)
    y, h = R.norm(x, w, r, 1e-5)
    got = sv.add_norm(x, w, r, eps=1e-5, e4m3=out == "e4m3", dtype=torch.float32 if out == "f32" else None)
    if r is not None:
        s = got[-1]
        assert s.dtype == r.dtype and s.shape == x.shape
        half = 2.0 ** -8 if rt == "bfloat16" else 0
        assert ((s.double() - h).abs() <= h.abs() * (half + 2.0 ** -23)).all()
    # the sum of squares is off by 96 roundings of 2^-24 at most (80 terms of a thread in turn, then trees),
    # half of that after the root, and a root of 2^-22 and four roundings more
    slack = 2.0 ** -18
    if out == "e4m3":
        R.check_e4m3(got[0], got[1], y, slack=slack)
        assert got[1].stride(0) == 1 or rows == 1
    else:
        z = got if r is None else got[0]
        half = 2.0 ** -8 if out == "bf16" else 0
        assert z.dtype == (torch.bfloat16 if out == "bf16" else torch.float32)
        assert ((z.double() - y).abs() <= y.abs() * (half + slack)).all()


def test_add_norm_in_place_strided_and_shapes(sv):
    g = gen(1)
    big = torch.randn((6, 5, 3, 256), generator=g, device="cuda").to(torch.bfloat16)
    x = big[:, :, 1]                                          # [6, 5, 256], rows 768 apart
    stream = torch.randn((6, 5, 512), generator=g, device="cuda")[:, :, 256:]
    before = stream.clone()
    y, h = R.norm(x.reshape(30, 256), None, before.reshape(30, 256), 1e-6)
    q, sc, s = sv.add_norm(x, None, stream, e4m3=True, sum_out=stream)
    assert s.data_ptr() == stream.data_ptr() and q.shape == x.shape and sc.shape == (6, 5, 2)
    assert ((stream.reshape(30, 256).double() - h).abs() <= h.abs() * 2.0 ** -23).all()
    R.check_e4m3(q.reshape(30, 256), sc.reshape(30, 2), y)
    # of x itself
    z = x.clone()
    y2, s2 = sv.add_norm(z, None, z.clone(), sum_out=z)
    assert s2.data_ptr() == z.data_ptr() and torch.equal(z, (x.float() * 2).to(torch.bfloat16))


@pytest.mark.parametrize("dim", [256, 40000])
def test_add_norm_long_rows_in_place(sv, dim):
    g = gen(dim)
    x = torch.randn((4, dim), generator=g, device="cuda").to(torch.bfloat16)
    r = torch.randn((4, dim), generator=g, device="cuda").to(torch.bfloat16)
    want, s = sv.add_norm(x, None, r)
    got, t = sv.add_norm(x, None, r, sum_out=r)
    assert torch.equal(want, got) and torch.equal(s, t) and torch.equal(t, r)


def test_add_norm_zero_rows_and_odd_values(sv):
    assert sv.add_norm(torch.zeros((0, 64), dtype=torch.bfloat16, device="cuda")).shape == (0, 64)
    x = torch.zeros((3, 256), device="cuda")
    q, sc = sv.add_norm(x, e4m3=True)
    assert (q.float() == 0).all() and ((sc.double() - 1e-20 / 448).abs() <= 1e-20 / 448 * 2.0 ** -22).all()
    x[1, 5] = float("inf")
    x[2, 200] = float("nan")
    y = sv.add_norm(x, dtype=torch.float32)
    assert (y[0] == 0).all() and y[2].isnan().all() and y[1, 5].isnan()
    # the far ends of the range: mean squares that underflow leave eps, of 1e18 they hold
    y = sv.add_norm(torch.full((1, 128), 1e-30, device="cuda"), dtype=torch.float32)
    assert ((y.double() - 1e-27).abs() <= 1e-27 * 2.0 ** -18).all()
    y = sv.add_norm(torch.full((1, 128), 1e18, device="cuda"), dtype=torch.float32)
    assert ((y.double() - 1).abs() <= 2.0 ** -20).all()


# ---- gated activation, rounding ----------------------------------------------------------
@pytest.mark.parametrize("weighted", [False, True])
def test_add_norm_to_8_bits_small_blocks_and_odd_values(sv, weighted):
    """Blocks under the least scale, and what is not finite, beside ordinary ones."""
    g = gen(7)
    x = torch.randn((5, 640), generator=g, device="cuda")
    x[:, 128:256] *= 1e-21
    x[:, 256:384] *= 3e-23
    x[:, 384:512] = 0
    w = (torch.rand(640, generator=g, device="cuda") + 0.5).to(torch.bfloat16) if weighted else None
    R.check_e4m3(*sv.add_norm(x, w, e4m3=True), R.norm(x, w, None, 1e-6)[0], slack=2.0 ** -18)
    want = sv.add_norm(x, w, e4m3=True)
    x[1, 5], x[3, 630] = float("inf"), float("nan")
    q, sc = sv.add_norm(x, w, e4m3=True)
    ok = [0, 2, 4]
    assert torch.equal(q[ok].float(), want[0][ok].float()) and torch.equal(sc[ok], want[1][ok])
    assert q[3].float().isnan().all() and q[1, 5].float().isnan() and (q[1].float().nan_to_num() == 0).all()


@pytest.mark.parametrize("rows,dim", [(1, 16), (7, 64), (3, 144), (33, 1008), (7, 12288), (129, 2048)])
@pytest.mark.parametrize("kind", ["silu", "gelu"])
@pytest.mark.parametrize("xt", ["bfloat16", "float32"])
@pytest.mark.parametrize("out", ["bf16", "f32", "e4m3"])
def test_gated_act(sv, rows, dim, kind, xt, out):
    g = gen(rows + dim)
    x = (3 * torch.randn((rows, 2 * dim), generator=g, device="cuda")).to(getattr(torch, xt))
    gate, up = x.chunk(2, -1)
    y = R.act(gate, up, kind)
    args = (gate, up) if dim == 144 else (x,)
    got = sv.gated_act(*args, act=kind, e4m3=out == "e4m3", dtype=torch.float32 if out == "f32" else None)
    # e^-t is off by 2 + 1.16 |t| steps of fp32 and more, t up to 3 |gate| here (for gate in 15: 50 steps), where the
    # logistic function passes that on times less than 1: |up| gate 2^-17
    off = gate.double().abs() * up.double().abs() * 2.0 ** -17
    if out == "e4m3":
        R.check_e4m3(got[0], got[1], y, slack=2.0 ** -16)
    else:
        half = 2.0 ** -8 if out == "bf16" else 0
        assert ((got.double() - y).abs() <= y.abs() * half + off + 1e-30).all()


def test_gated_act_ends_of_the_range(sv):
    gate = torch.tensor([0.0, -0.0, 90.0, -90.0, 1e30, -1e30, 3e38, -3e38], device="cuda")[None]
    up = torch.ones((1, 8), device="cuda")
    for kind in ("silu", "gelu"):
        y = sv.gated_act(gate, up, act=kind, dtype=torch.float32)[0]
        assert (y[[2, 4, 6]] == gate[0, [2, 4, 6]]).all() and (y[[0, 1, 3, 5, 7]].abs() < 1e-30).all()


@pytest.mark.parametrize("rows,dim", [(1, 16), (5, 128), (130, 144), (127, 4096), (257, 1040), (1, 20000)])
@pytest.mark.parametrize("xt", ["bfloat16", "float32"])
@pytest.mark.parametrize("high", [1, 128])
def test_quantize(sv, rows, dim, xt, high):
    x = (0.02 * torch.randn((rows, dim), generator=gen(rows), device="cuda")).to(getattr(torch, xt))
    x[rows // 2, dim // 2] = 3.0
    q, sc = sv.quantize_e4m3(x, block_rows=high)
    R.check_e4m3(q, sc, x.double(), high, slack=2.0 ** -23)
    # the formula in fp32, element for element
    top = R.block_top(x.float(), high).clamp_min(1e-20)
    most = torch.full_like(top, 448)                          # (by or of a number, torch multiplies with a reciprocal)
    f = (most / top).repeat_interleave(high, 0)[:rows].repeat_interleave(128, 1)[:, :dim]
    assert torch.equal(q.view(torch.uint8), (x.float() * f).to(torch.float8_e4m3fn).view(torch.uint8))
    assert torch.equal(sc, top / most)


@pytest.mark.parametrize("high", [1, 128])
def test_quantize_odd_values(sv, high):
    x = torch.zeros((4, 384), device="cuda")
    x[0, 3], x[0, 4] = float("nan"), 2.0
    x[1, 130], x[1, 131] = float("inf"), 1.0
    q, sc = sv.quantize_e4m3(x, block_rows=high)
    v = R.value(q, sc, high)
    assert v[0, 3].isnan() and abs(v[0, 4] - 2) <= 2.0 ** -20 and v[1, 130].isnan() and v[1, 131].isnan()
    assert (v[2:, 256:] == 0).all() and (v[0, 5:128] == 0).all()


# ---- product ------------------------------------------------------------------------------
def check(sv, seed, M, N, K, dtype, **kw):
    x, xs, w, ws = R.problem(seed, M, N, K)
    got = sv.matmul_e4m3(x, xs, w, ws, dtype=dtype, **kw)
    ref, mags = R.matmul(x, xs, w, ws)
    assert got.shape == (M, N) and got.dtype == dtype
    err, bound = (got.double() - ref).abs(), R.matmul_bound(ref, mags, K, dtype)
    assert (err <= bound).all(), ((err / bound).max(), (err > bound).nonzero()[:8].tolist())
    return got


ROWS = [1, 2, 7, 15, 16, 17, 31, 33, 64, 65, 100, 127, 128, 129, 200, 256, 257, 300, 511, 640]


@pytest.mark.parametrize("M", ROWS)
@pytest.mark.parametrize("N,K", [(1, 16), (7, 128), (64, 144), (128, 256), (129, 1040), (1000, 384), (384, 4096)])
def test_matmul(sv, M, N, K):
    check(sv, M + N + K, M, N, K, torch.float32 if (M + N) % 2 else torch.bfloat16)


@pytest.mark.parametrize("M,N,K", [(1, 6144, 4096), (8, 4096, 12288), (512, 6144, 4096), (1152, 4096, 2048), (77, 151936, 256),
                                   (2500, 1111, 528), (130, 40000, 272), (64, 20000, 16384), (4, 128, 30000)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_matmul_large(sv, M, N, K, dtype):
    check(sv, N, M, N, K, dtype)


@pytest.mark.parametrize("M,N,K", [(70, 64, 128), (70, 64, 400), (100, 130, 1168), (257, 500, 1680), (300, 200, 2000), (300, 1900, 5200),
                                   (600, 1000, 16400), (520, 4700, 1296), (1152, 2000, 9008), (90, 4800, 1040)])
def test_matmul_odd_numbers_of_blocks(sv, M, N, K):
    """Steps of two blocks, parts of tiles and clusters whose blocks come out odd."""
    check(sv, M + N, M, N, K, torch.float32)


@pytest.mark.parametrize("M", [5, 120, 140])
def test_matmul_accumulates_in_fp32(sv, M):
    """One large product and many small ones of the other scale: 14 bits of a sum would lose them."""
    K, N = 128, 128
    x = torch.full((M, K), 1.0, device="cuda").to(torch.float8_e4m3fn)
    w = torch.full((N, K), 2.0 ** -6, device="cuda").to(torch.float8_e4m3fn)
    w[:, 5] = 448.0
    x[:, 5] = 64.0
    one = torch.ones((1, M), device="cuda").t()
    got = sv.matmul_e4m3(x, one, w, torch.ones((1, 1), device="cuda"), dtype=torch.float32)
    want = 448.0 * 64 + 127 / 64
    assert ((got.double() - want).abs() <= 128 * want * 2.0 ** -24).all() and (got - want).abs().max() < 0.25


@pytest.mark.parametrize("M", [9, 40, 100, 300])
def test_matmul_strides_shapes_and_nan(sv, M):
    """Rows and outputs with strides of their own, K that is no multiple of 16, leading dimensions; NaN
    stays in its row and in its column."""
    K, N = 200, 264
    x, xs, w, ws = R.problem(M, M, N, K)
    bigx = torch.full((M, 272), 0x7f, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)     # NaN around
    bigw = torch.full((N, 208), 0x7f, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    bigx.view(torch.uint8)[:, 16:16 + K] = x.view(torch.uint8)
    bigw.view(torch.uint8)[:, :K] = w.view(torch.uint8)
    out = torch.full((M, N + 5), -7.0, device="cuda")
    got = sv.matmul_e4m3(bigx[:, 16:16 + K], xs, bigw[:, :K], ws, dtype=torch.float32, out=out[:, 3:3 + N])
    assert got.data_ptr() == out[:, 3:].data_ptr() and (out[:, :3] == -7).all() and (out[:, 3 + N:] == -7).all()
    ref, mags = R.matmul(x, xs, w, ws)
    assert ((got.double() - ref).abs() <= R.matmul_bound(ref, mags, K, torch.float32)).all()
    if M % 3 == 0:
        many = sv.matmul_e4m3(bigx[:, 16:16 + K].unflatten(0, (3, M // 3)), xs.unflatten(0, (3, M // 3)), bigw[:, :K], ws, dtype=torch.float32)
        assert many.shape == (3, M // 3, N) and torch.equal(many.reshape(M, N), got)
    bigx.view(torch.uint8)[M // 2, 20] = 0x7f
    bigw.view(torch.uint8)[7, 20] = 0x7f
    bad = sv.matmul_e4m3(bigx[:, 16:16 + K], xs, bigw[:, :K], ws, dtype=torch.float32)
    nan = torch.zeros((M, N), dtype=torch.bool, device="cuda")
    nan[M // 2], nan[:, 7] = True, True
    assert torch.equal(bad.isnan(), nan) and torch.equal(bad[~nan], got[~nan])


@pytest.mark.parametrize("M", [2, 33, 70, 270])
@pytest.mark.parametrize("K", [1, 3, 17, 129])
def test_matmul_short_contractions(sv, M, K):
    x, xs, w, ws = R.problem(M + K, M, 90, K)
    rows = []
    for t in (x, w):                                          # NaN from K on
        wide = torch.full((t.shape[0], 144), 0x7f, dtype=torch.uint8, device="cuda")
        wide[:, :K] = t.view(torch.uint8)
        rows.append(wide.view(torch.float8_e4m3fn)[:, :K])
    got = sv.matmul_e4m3(rows[0], xs, rows[1], ws, dtype=torch.float32)
    ref, mags = R.matmul(x, xs, w, ws)
    assert ((got.double() - ref).abs() <= R.matmul_bound(ref, mags, K, torch.float32)).all()


@pytest.mark.parametrize("M", [5, 64, 100, 300])
@pytest.mark.parametrize("N,stride,at", [(262, 264, 0), (263, 272, 0), (261, 268, 4), (130, 132, 2), (129, 131, 1), (70, 1000, 8)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_matmul_into_wider_rows(sv, M, N, stride, at, dtype):
    """Rows of an output that is a slice: whatever their stride's alignment, nothing beside them is written."""
    p = R.problem(N, M, N, 400)
    want = sv.matmul_e4m3(*p, dtype=dtype)
    room = torch.full((M + 2, stride), -7.0, device="cuda", dtype=dtype)
    got = sv.matmul_e4m3(*p, dtype=dtype, out=room[1:-1, at:at + N])
    assert torch.equal(got, want)
    room[1:-1, at:at + N] = -7
    assert (room == -7).all()


@pytest.mark.parametrize("M", [3, 100, 700])
def test_matmul_repeats_itself(sv, M):
    x, xs, w, ws = R.problem(M, M, 1500, 2064)
    first = sv.matmul_e4m3(x, xs, w, ws, dtype=torch.float32)
    for _ in range(5):
        assert torch.equal(first, sv.matmul_e4m3(x, xs, w, ws, dtype=torch.float32))


@pytest.mark.parametrize("M,N,K", [(64, 20000, 4096), (32, 20000, 4096), (16, 20000, 4096), (64, 1000, 4096), (100, 700, 4096),
                                   (512, 6144, 4096), (700, 1000, 16384)])
def test_matmul_agrees_with_itself_over_many_runs(sv, M, N, K):
    """Enough runs, with the memory busy now and then, for a stage that is written again too early."""
    p = R.problem(M, M, N, K)
    first = sv.matmul_e4m3(*p, dtype=torch.float32)
    other = torch.empty(32 << 20, device="cuda")
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(400):
        if i % 3 == 0:
            other.fill_(i)
        differ += (sv.matmul_e4m3(*p, dtype=torch.float32) != first).sum()
    assert int(differ) == 0


def test_matmul_empty(sv):
    x, xs, w, ws = R.problem(0, 4, 32, 64)
    assert sv.matmul_e4m3(x[:0], xs[:0], w, ws).shape == (0, 32)
    assert sv.matmul_e4m3(x, xs, w[:0], ws[:0]).shape == (4, 0)


# ---- all of it -----------------------------------------------------------------------------
@pytest.mark.parametrize("rows", [1, 24, 180])
def test_feed_forward(sv, rows):
    """Norm, gate and up, activation, down, residual, as a layer runs them, against 64 bits with the
    same 8-bit weights: rows are rounded to e4m3 three times on the way."""
    g = gen(rows)
    dim, wide = 512, 1024
    x = torch.randn((rows, dim), generator=g, device="cuda").to(torch.bfloat16)
    r = torch.randn((rows, dim), generator=g, device="cuda").to(torch.bfloat16)
    nw = (torch.rand(dim, generator=g, device="cuda") + 0.5).to(torch.bfloat16)
    gu = (torch.randn((2 * wide, dim), generator=g, device="cuda") * dim ** -0.5).to(torch.bfloat16)
    dn = (torch.randn((dim, wide), generator=g, device="cuda") * wide ** -0.5).to(torch.bfloat16)
    gu8, dn8 = sv.quantize_e4m3(gu, block_rows=128), sv.quantize_e4m3(dn, block_rows=128)
    q, sc, h = sv.add_norm(x, nw, r, e4m3=True)
    a = sv.gated_act(sv.matmul_e4m3(q, sc, *gu8), e4m3=True)
    y, h2 = sv.add_norm(sv.matmul_e4m3(*a, *dn8), None, h)
    ny, nh = R.norm(x, nw, r, 1e-6)
    gate, up = (ny @ R.value(*gu8, 128).t()).chunk(2, -1)
    down = R.act(gate, up, "silu") @ R.value(*dn8, 128).t()
    # rms of the roundings: e4m3 2^-4 / sqrt 3 of a value twice (rows, activations), bf16 on top: each product
    # averages them over its terms, so about 0.036 * 2 of the result's rms; its largest of 1e5 values 5 times that
    err = (h2.double() - (nh + down)).abs()
    assert err.square().mean().sqrt() <= 0.1 * down.square().mean().sqrt() + 2.0 ** -8 * nh.square().mean().sqrt()
    assert err.max() <= 0.6 * down.square().mean().sqrt() + 2.0 ** -7 * nh.abs().max()
    want = R.norm(h2, None, None, 1e-6)[0]
    assert ((y.double() - want).abs() <= want.abs() * 2.0 ** -6 + 2.0 ** -8).all()

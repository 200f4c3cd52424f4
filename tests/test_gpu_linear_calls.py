"""How the calls of the target model's dense side are made: captured and replayed, on several streams, with
workspaces of any contents, on inputs that a kernel has just written, past 32-bit offsets, with waits that
run out."""
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


# few rows with one CTA and with clusters; clusters of pairs; whole tiles; tiles shared by pairs, of two
# widths
SHAPES = [(3, 400, 128), (9, 300, 4096), (64, 1000, 2048), (100, 700, 1024), (300, 128, 16384), (700, 5000, 1040), (600, 1000, 16384),
          (1100, 2600, 12288)]


def feed_forward(sv, seed, rows, dim, wide):
    """Inputs and a pass through all four calls, as a layer makes it."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def r(*shape):
        return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)
    x, res, w = r(rows, dim), r(rows, dim), r(dim)
    up, down = (sv.quantize_e4m3(r(*s) * s[1] ** -0.5, block_rows=128) for s in ((2 * wide, dim), (dim, wide)))

    def run():
        q, s, h = sv.add_norm(x, w, res, e4m3=True)
        a = sv.gated_act(sv.matmul_e4m3(q, s, *up), e4m3=True)
        return sv.add_norm(sv.matmul_e4m3(*a, *down), w, h)
    return (x, res, w), run


@pytest.mark.parametrize("rows,dim,wide", [(1, 256, 512), (40, 1024, 640), (300, 512, 1024), (700, 4096, 8192)])
def test_captured_and_replayed(sv, rows, dim, wide):
    """A captured pass, replayed on new contents of its inputs, gives what calls on them give."""
    ins, run = feed_forward(sv, rows, rows, dim, wide)
    want = [t.clone() for t in run()]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        held = run()
    for turn in range(3):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want)), turn
        for t in ins[:2]:
            t.mul_(0.75)
        want = [t.clone() for t in run()]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_workspaces_of_any_contents(sv, M, N, K):
    p = R.problem(M, M, N, K)
    want = sv.matmul_e4m3(*p, dtype=torch.float32)
    need = sv.load_library().spec_matmul_workspace_size(M, N, K)
    for fill in (0, 0xff, 0x5a, None):
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        if fill is None:
            ws.random_(0, 256)
        else:
            ws.fill_(fill)
        ws[:256] = 0
        for _ in range(2):
            assert torch.equal(want, sv.matmul_e4m3(*p, dtype=torch.float32, workspace=ws))
        assert (ws[:256] == 0).all()
    w = sv.Workspace()
    assert torch.equal(want, sv.matmul_e4m3(*p, dtype=torch.float32, workspace=w)) and w.read_error() == 0


def test_one_workspace_for_calls_of_all_kinds(sv):
    w = sv.Workspace()
    z = torch.randn((3, 50257), device="cuda")
    tok = torch.zeros(3, dtype=torch.int32, device="cuda")
    lp = [t.clone() for t in sv.token_logprobs(z, tok, 4)]
    for M, N, K in SHAPES:
        p = R.problem(M, M, N, K)
        want = sv.matmul_e4m3(*p, dtype=torch.float32)
        assert torch.equal(want, sv.matmul_e4m3(*p, dtype=torch.float32, workspace=w))
        assert all(torch.equal(a, b) for a, b in zip(lp, sv.token_logprobs(z, tok, 4, workspace=w)))
        assert torch.equal(want, sv.matmul_e4m3(*p, dtype=torch.float32, workspace=w))
    assert w.read_error() == 0


def test_calls_on_two_streams_at_once(sv):
    jobs = [feed_forward(sv, i, rows, 1024, 2048)[1] for i, rows in enumerate((500, 12, 300))]
    want = [[t.clone() for t in j()] for j in jobs]
    streams = [torch.cuda.Stream() for _ in jobs]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for j, s in zip(jobs, streams):
            with torch.cuda.stream(s):
                got.append(j())
    torch.cuda.synchronize()
    for i, r in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(r, want[i % 3]))
    # the stream as an argument, from another current one
    q, s, h = sv.add_norm(torch.ones((4, 256), device="cuda", dtype=torch.bfloat16), None, torch.ones((4, 256), device="cuda"), e4m3=True,
                          stream=streams[0])
    streams[0].synchronize()
    assert (h == 2).all() and (q.float() == 448).all()


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_inputs_written_by_the_kernel_before(sv, M, N, K):
    """Rows, scales and weights rewritten on the stream just before every call, without a wait."""
    sets = [R.problem(M + i, M, N, K) for i in range(3)]
    want = [sv.matmul_e4m3(*p, dtype=torch.float32) for p in sets]
    x, xs, w, ws = (t.clone() for t in sets[0])
    xs = R.scales(torch.Generator(device="cuda"), M, xs.shape[1])
    out = []
    for i in range(9):
        for a, b in zip((x, w), (sets[i % 3][0], sets[i % 3][2])):
            a.view(torch.uint8).copy_(b.view(torch.uint8))
        xs.copy_(sets[i % 3][1])
        ws.copy_(sets[i % 3][3])
        out.append(sv.matmul_e4m3(x, xs, w, ws, dtype=torch.float32))
    assert all(torch.equal(o, want[i % 3]) for i, o in enumerate(out))


def test_offsets_past_32_bits(sv):
    rows, dim = 270000, 8192                                   # 2.2e9 elements
    x = torch.zeros((rows, dim), dtype=torch.bfloat16, device="cuda")
    last = torch.randn((3, dim), device="cuda").to(torch.bfloat16)
    x[-3:] = last
    q, sc = sv.quantize_e4m3(x)
    R.check_e4m3(q[-3:], sc[-3:], last.double(), slack=2.0 ** -22)
    q, sc = sv.quantize_e4m3(x, block_rows=128)
    R.check_e4m3(q[rows // 128 * 128:], sc[-1:], torch.cat([torch.zeros((rows % 128 - 3, dim), device="cuda"), last]).double(), 128, slack=2.0 ** -22)
    q, sc, h = sv.add_norm(x, None, x, e4m3=True)
    assert torch.equal(h[-3:], (last.float() * 2).to(torch.bfloat16))
    R.check_e4m3(q[-3:], sc[-3:], R.norm(last, None, last, 1e-6)[0])
    y = sv.gated_act(x)
    ref = R.act(*last.chunk(2, -1), "silu")
    assert ((y[-3:].double() - ref).abs() <= ref.abs() * 2.0 ** -8 + last.abs().max() ** 2 * 2.0 ** -17).all()
    del h, x, y
    # a weight of 2.2e9 elements (q, rows of another's scales) times 2 and 200 rows, an output of 2.4e9
    g = torch.Generator(device="cuda").manual_seed(1)
    ws = torch.full(((rows + 127) // 128, dim // 128), 1.0 / 448, device="cuda")
    w = q
    for M in (2, 200):
        a, s = R.rand_e4m3(g, M, dim), R.scales(g, M, dim // 128)
        got = sv.matmul_e4m3(a, s, w, ws, dtype=torch.float32)
        ref, mags = R.matmul(a, s, w[-200:], ws[-2:])         # (one scale for all)
        assert ((got[:, -200:].double() - ref).abs() <= R.matmul_bound(ref, mags, dim, torch.float32)).all()
    del w, q, got
    M, N = 20000, 121000
    a, s, b, t = R.problem(5, M, N, 128)
    got = sv.matmul_e4m3(a, s, b, t)
    ref, mags = R.matmul(a[-300:], s[-300:], b[-(N % 128) - 128:], t[-2:])
    assert ((got[-300:, -(N % 128) - 128:].double() - ref).abs() <= R.matmul_bound(ref, mags, 128, torch.bfloat16)).all()


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_wait_limit_zero_times_out_then_recovers(sv, M, N, K):
    p = R.problem(M, M, N, K)
    want = sv.matmul_e4m3(*p, dtype=torch.float32)
    w = sv.Workspace()
    sv.matmul_e4m3(*p, workspace=w)
    assert w.read_error() == 0
    sv.spec_verify_set_wait_limit(0)
    try:
        bad = sv.matmul_e4m3(*p, dtype=torch.float32, workspace=w)
        torch.cuda.synchronize()
    finally:
        sv.spec_verify_set_wait_limit(sv.spec_verify_default_wait_limit())
    assert w.read_error() == sv.SPEC_DEVERR_TIMEOUT and bad.isnan().all()
    assert torch.equal(want, sv.matmul_e4m3(*p, dtype=torch.float32, workspace=w)) and w.read_error() == 0


def test_refusals(sv):
    x = torch.zeros((4, 256), dtype=torch.bfloat16, device="cuda")
    q, s = sv.quantize_e4m3(x)
    w, ws = sv.quantize_e4m3(x, block_rows=128)
    for call, error in [
        (lambda: sv.add_norm(x.half()), TypeError), (lambda: sv.add_norm(x, x[0].float()), TypeError),
        (lambda: sv.add_norm(x, x[0, :128]), ValueError), (lambda: sv.add_norm(x, None, x[:2]), ValueError),
        (lambda: sv.add_norm(x, None, sum_out=x), ValueError), (lambda: sv.add_norm(x, None, x, sum_out=x.float()), TypeError),
        (lambda: sv.add_norm(x.t()), ValueError), (lambda: sv.add_norm(x[:, :252].contiguous()), sv.SpecVerifyError),
        (lambda: sv.add_norm(x[:, 4:132]), sv.SpecVerifyError), (lambda: sv.add_norm(x.unflatten(0, (2, 2)).transpose(0, 1)), ValueError),
        (lambda: sv.gated_act(x, x.float()), TypeError), (lambda: sv.gated_act(x, x[:, :128]), ValueError),
        (lambda: sv.gated_act(x[:, :255].contiguous()), ValueError), (lambda: sv.quantize_e4m3(x, block_rows=64), ValueError),
        (lambda: sv.quantize_e4m3(x.unflatten(0, (2, 2)), block_rows=128), ValueError), (lambda: sv.quantize_e4m3(q), TypeError),
        (lambda: sv.matmul_e4m3(x, s, w, ws), TypeError), (lambda: sv.matmul_e4m3(q, s, w[:, :128], ws), ValueError),
        (lambda: sv.matmul_e4m3(q, s[:, :1], w, ws), ValueError), (lambda: sv.matmul_e4m3(q, s.contiguous(), w, ws), ValueError),
        (lambda: sv.matmul_e4m3(q, s, w, ws[:, :1]), ValueError), (lambda: sv.matmul_e4m3(q, s.double(), w, ws), TypeError),
        (lambda: sv.matmul_e4m3(q, s, w, ws, out=x), ValueError), (lambda: sv.matmul_e4m3(q, s, w, ws, dtype=torch.float16), TypeError),
        (lambda: sv.matmul_e4m3(q, s, w, ws, out=torch.empty((4, 4), device="cuda")), TypeError),
        (lambda: sv.matmul_e4m3(q, s, w, ws, workspace=torch.empty(16, dtype=torch.uint8, device="cuda")), sv.SpecVerifyError),
        (lambda: sv.matmul_e4m3(q[1:, 8:136], s[1:, :1], w[:, :128], ws[:, :1]), sv.SpecVerifyError),
    ]:
        with pytest.raises(error):
            call()
    assert sv.matmul_e4m3(q, s, w, ws).shape == (4, 4)


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_captured_products(sv, M, N, K):
    """A captured product replayed on contents that change: shared tiles' tickets are counted anew in every
    replay."""
    sets = [R.problem(M + 7 * i, M, N, K) for i in range(2)]
    want = [sv.matmul_e4m3(*p, dtype=torch.float32) for p in sets]
    x, xs, w, ws = R.problem(M, M, N, K)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        held = sv.matmul_e4m3(x, xs, w, ws, dtype=torch.float32)
    for turn in range(4):
        y, ys, v, vs = sets[turn % 2]
        x.view(torch.uint8).copy_(y.view(torch.uint8))
        w.view(torch.uint8).copy_(v.view(torch.uint8))
        xs.copy_(ys)
        ws.copy_(vs)
        held.fill_(-1)
        graph.replay()
        assert torch.equal(held, want[turn % 2]), turn


@pytest.mark.parametrize("lead,strides", [((5,), (0,)), ((4, 3), (0, 0)), ((4, 3), (256, 0)), ((4, 3), (0, 256))])
def test_expanded_rows(sv, lead, strides):
    """One row in place of many: read as such, refused where rows lie otherwise than one stride apart, as an output and by
    the product, which takes rows of their own."""
    store = torch.randn((64, 256), device="cuda").to(torch.bfloat16)
    x = store.as_strided(lead + (256,), strides + (1,))
    shared = not any(strides)
    for call in (lambda t: sv.add_norm(t, None, t), lambda t: sv.gated_act(t), lambda t: sv.quantize_e4m3(t)):
        if shared:
            assert all(torch.equal(a, b) for a, b in zip(call(x), call(x.contiguous())))
        else:
            with pytest.raises(ValueError, match="one stride apart"):
                call(x)
    with pytest.raises((ValueError, sv.SpecVerifyError)):
        sv.add_norm(x.contiguous(), None, x.contiguous(), sum_out=x)
    q, s = sv.quantize_e4m3(x.contiguous())
    w, ws = sv.quantize_e4m3(store, block_rows=128)
    q1, s1 = sv.quantize_e4m3(store)
    q1 = q1.as_strided(lead + (256,), strides + (1,))
    s1 = s1.as_strided(lead + (2,), tuple(d // 256 for d in strides) + (s1.stride(-1),))
    for a, b in ((q1, s), (q, s1)):
        with pytest.raises((ValueError, sv.SpecVerifyError)):
            sv.matmul_e4m3(a, b, w, ws)
    with pytest.raises((ValueError, sv.SpecVerifyError)):
        sv.matmul_e4m3(q, s, w[:1], ws, out=store.as_strided(lead + (1,), strides + (1,)))
    with pytest.raises((ValueError, sv.SpecVerifyError)):
        sv.matmul_e4m3(q, s, q1[0, :1].expand(8, 256) if q1.dim() == 3 else q1[:1].expand(8, 256), ws)

"""Token log-probabilities, entropies and top alternatives against the 64-bit form
(tests/kv_ref.py)."""
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


def check(sv, z, tok, K, T, **kw):
    """z on the CPU, as the kernel reads it.  Exponents' arguments are off by a few u32 |a| and the
    terms that matter have |a| < 40 (in powers of two), 2^x by 2 u32: sums are within 2^-18 of
    themselves, an entropy's inner sum within that of sum p |a| <= H + ln V."""
    lp, ent, ti, tl = sv.token_logprobs(z.cuda(), tok.cuda(), K, temperature=T, **kw)
    l, e, i, t = R.logprobs(z, tok, K, T)
    tol = 2.0 ** -18 + 2.0 ** -22 * l.abs()
    fin = torch.isfinite(l)
    assert torch.equal(torch.isfinite(lp.cpu()), fin)
    assert ((lp.cpu().double() - l).abs()[fin] <= tol[fin]).all()
    assert ((ent.cpu().double() - e).abs() <= 2.0 ** -18 * (1 + e + math.log(z.shape[1]))).all()
    if K:
        assert torch.equal(ti.cpu().long(), i)
        fin = torch.isfinite(t.float())                          # past fp32's range: -inf
        assert torch.equal(torch.isfinite(tl.cpu()), fin)
        assert ((tl.cpu().double() - t).abs()[fin] <= 2.0 ** -18 + 2.0 ** -22 * t.abs()[fin]).all()
    else:
        assert ti is None and tl is None


def rows(seed, R_, V, f32, sigma=3.0):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn((R_, V), generator=g) * sigma
    tok = torch.randint(0, V, (R_,), generator=g).to(torch.int32)
    return (z if f32 else z.to(torch.bfloat16)), tok


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("R_,V", [(1, 1), (3, 2), (5, 7), (2, 1000), (4, 1001), (3, 16384), (3, 16385), (7, 32767),
                                  (2, 50257), (1, 151936), (9, 8191), (1, 131075)])
@pytest.mark.parametrize("K", [0, 1, 5])
def test_rows_of_every_alignment(sv, f32, R_, V, K):
    z, tok = rows(V + K, R_, V, f32)
    check(sv, z, tok, K, 0.7)


@pytest.mark.parametrize("K", [1, 2, 3, 4, 8])
@pytest.mark.parametrize("T", [1.0, 0.05, 30.0])
def test_temperatures_and_list_lengths(sv, K, T):
    for f32 in (False, True):
        z, tok = rows(K, 6, 20011, f32)
        check(sv, z, tok, K, T)


def test_many_rows(sv):
    z, tok = rows(3, 700, 5003, False)
    check(sv, z, tok, 4, 1.0)


def test_ties_take_the_lowest_index(sv):
    """Equal logits everywhere, two values, and signed zeros."""
    for f32 in (False, True):
        V = 40009
        dt = torch.float32 if f32 else torch.bfloat16
        z = torch.zeros((4, V), dtype=dt)
        z[1, ::2] = -0.0
        z[2, 17::1000] = 2.0
        z[3] = torch.arange(V).remainder(3).to(dt)
        check(sv, z, torch.tensor([0, V - 1, 17, 2], dtype=torch.int32), 8, 1.0)


@pytest.mark.parametrize("f32", [False, True])
def test_masked_logits(sv, f32):
    """-inf, the type's lowest value, and rows with fewer finite logits than the list is long."""
    V = 30001
    z, tok = rows(8, 6, V, f32)
    low = torch.finfo(z.dtype).min
    z[0, 100:] = -math.inf
    z[1, 2:] = -math.inf
    z[2, :-1] = -math.inf
    z[3, 5:] = low
    z[4, ::3] = -math.inf
    tok = torch.tensor([5, 0, V - 1, 3, 3, 10], dtype=torch.int32)
    check(sv, z, tok, 8, 0.9)


@pytest.mark.parametrize("f32", [False, True])
def test_rows_masked_with_the_lowest_value(sv, f32):
    """Whole chunks, and whole rows, of the type's lowest finite value or beside -inf."""
    V = 50000
    z, tok = rows(13, 4, V, f32)
    low = torch.finfo(z.dtype).min
    z[0, 3000:] = low
    z[1] = low
    z[2] = low
    z[2, ::2] = -math.inf
    z[3, :-5] = -math.inf
    check(sv, z, torch.tensor([5, 7, 1, V - 2], dtype=torch.int32), 8, 1.0)


@pytest.mark.parametrize("f32", [False, True])
def test_top_tokens_in_few_chunks_and_in_many(sv, f32):
    """Sorted rows (all of the top in one chunk), rows of few values, and a long row."""
    V = 100003
    dt = torch.float32 if f32 else torch.bfloat16
    z = torch.empty((4, V), dtype=dt)
    z[0] = torch.linspace(-9, 9, V).to(dt)
    z[1] = torch.linspace(9, -9, V).to(dt)
    z[2] = (torch.arange(V) % 7).to(dt)
    z[3] = torch.where(torch.arange(V) % 5000 == 4999, 3.0, -2.0).to(dt)
    check(sv, z, torch.tensor([V - 1, 0, 6, 4999], dtype=torch.int32), 8, 1.0)
    z, tok = rows(14, 2, 1500007, f32)
    check(sv, z, tok, 7, 1.0)


def test_large_logits_and_small_temperatures(sv):
    z, tok = rows(9, 4, 9001, True)
    check(sv, z + 1000.0, tok, 3, 1.0)
    check(sv, z * 50, torch.argmax(z, 1).to(torch.int32), 3, 1.0)
    top = torch.argmax(z, 1).to(torch.int32)
    lp, ent, ti, tl = sv.token_logprobs(z.cuda(), top.cuda(), 2, temperature=1e-20)
    assert (lp == 0).all() and (ent == 0).all() and torch.equal(ti[:, 0].cpu(), top) and (tl[:, 0] == 0).all()


def test_bad_rows_are_marked_and_the_others_hold(sv):
    V = 5000
    z, tok = rows(10, 4, V, False)
    want = sv.token_logprobs(z.cuda(), tok.cuda(), 3)
    z[1] = -math.inf
    tok[2] = V
    tok[3] = -1
    ws = torch.zeros(sv.load_library().spec_logprobs_workspace_size(4, V, 3), dtype=torch.uint8, device="cuda")
    lp, ent, ti, tl = sv.token_logprobs(z.cuda(), tok.cuda(), 3, workspace=ws)
    st, code = sv.spec_verify_read_error(ws.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert st == 0 and code == sv.SPEC_DEVERR_TOKEN_RANGE | sv.SPEC_DEVERR_EMPTY_ROW
    assert lp[0] == want[0][0] and torch.isnan(lp[1:]).all()
    assert torch.isnan(ent[1]) and torch.equal(ent[[0, 2, 3]], want[1][[0, 2, 3]])
    assert (ti[1] == -1).all() and torch.isnan(tl[1]).all() and torch.equal(ti[[0, 2, 3]], want[2][[0, 2, 3]])


def test_streams_capture_and_repeats(sv):
    z, tok = rows(11, 64, 30000, False)
    zd, td = z.cuda(), tok.cuda()
    want = sv.token_logprobs(zd, td, 4)
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(3)]
    got = [sv.token_logprobs(zd, td, 4, stream=s) for _ in range(10) for s in side]
    torch.cuda.synchronize()
    for r in got:
        assert all(torch.equal(a, b) for a, b in zip(r, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = sv.token_logprobs(zd, td, 4)
    for _ in range(3):
        graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(held, want))
    zd.neg_()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(held, sv.token_logprobs(zd, td, 4)))


def test_shapes_and_refusals(sv):
    z, tok = rows(12, 6, 1000, False)
    a = sv.token_logprobs(z.cuda(), tok.cuda(), 2)
    b = sv.token_logprobs(z.cuda().view(2, 3, 1000), tok.cuda().view(2, 3), 2)
    assert b[0].shape == (2, 3) and b[2].shape == (2, 3, 2) and torch.equal(a[3].view(2, 3, 2), b[3])
    with pytest.raises(ValueError):
        sv.token_logprobs(z.cuda(), tok.cuda(), 9)
    with pytest.raises(ValueError):
        sv.token_logprobs(z.cuda(), tok.cuda()[:2], 2)
    with pytest.raises((TypeError, ValueError)):
        sv.token_logprobs(z.cuda(), tok.cuda().long(), 2)
    with pytest.raises(TypeError):
        sv.token_logprobs(z.cuda().half(), tok.cuda(), 2)
    with pytest.raises(sv.SpecVerifyError):
        sv.token_logprobs(z.cuda(), tok.cuda(), 2, temperature=0.0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,V,K", [(700, 8999, 0), (700, 8999, 1), (2600, 2001, 0), (30, 32001, 0), (610, 10300, 0)])
def test_many_middling_rows(sv, dtype, rows, V, K):
    """Rows of a few chunks, enough of them for the stream and too few for it."""
    g = torch.Generator().manual_seed(V + rows)
    z = (torch.randn(rows, V, generator=g) * 3).to(dtype)
    z[torch.rand(rows, V, generator=g) < 0.05] = -math.inf
    z[:, V // 3] = 1.0
    check(sv, z, torch.randint(0, V, (rows,), generator=g, dtype=torch.int32), K, 0.8)

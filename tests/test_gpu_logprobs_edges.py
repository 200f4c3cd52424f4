"""Token log-probabilities where something is out of the ordinary: a wait that runs out, the
largest temperatures, the package's own workspaces."""
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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("K", [0, 5])
def test_a_wait_that_runs_out_leaves_no_numbers(sv, dtype, K):
    """With the bounded waits set to give up at once, through a workspace that holds the sums of
    another call: every result is NaN (list tokens -1), the error word says why, and the next call
    is right again."""
    rows, V = 6, 151937
    g = torch.Generator(device="cuda").manual_seed(K)
    z = (torch.randn((rows, V), generator=g, device="cuda") * 3).to(dtype)
    tok = torch.arange(rows, dtype=torch.int32, device="cuda")
    ws = torch.zeros(sv.load_library().spec_logprobs_workspace_size(rows, V, K), dtype=torch.uint8, device="cuda")
    want = sv.token_logprobs(z, tok, K, workspace=ws)
    stream = torch.cuda.current_stream().cuda_stream
    torch.cuda.synchronize()
    assert sv.spec_verify_read_error(ws.data_ptr(), stream) == (0, 0)
    sv.spec_verify_set_wait_limit(0)
    try:
        got = sv.token_logprobs(z, tok, K, workspace=ws)
        torch.cuda.synchronize()
    finally:
        sv.spec_verify_set_wait_limit(sv.spec_verify_default_wait_limit())
    assert sv.spec_verify_read_error(ws.data_ptr(), stream) == (0, sv.SPEC_DEVERR_TIMEOUT)
    assert torch.isnan(got[0]).all() and torch.isnan(got[1]).all()
    if K:
        assert (got[2] == -1).all() and torch.isnan(got[3]).all()
    again = sv.token_logprobs(z, tok, K, workspace=ws)
    assert all(a is b is None or torch.equal(a, b) for a, b in zip(again, want))
    assert sv.spec_verify_read_error(ws.data_ptr(), stream) == (0, 0)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("V", [1000, 30001, 151937])
@pytest.mark.parametrize("T", [1e30, 1e36, 1e38, 3e38])
def test_masked_logits_at_the_largest_temperatures(sv, dtype, V, T):
    """A masked logit has no weight at any temperature; the others' are all but equal.  Tolerances
    as in test_gpu_logprobs.py."""
    g = torch.Generator().manual_seed(V)
    z = (torch.randn((4, V), generator=g) * 3).to(dtype)
    z[0, ::3] = -math.inf
    z[1, 5:] = -math.inf
    z[2, :V // 2] = -math.inf
    tok = torch.tensor([1, 4, V - 1, 0], dtype=torch.int32)
    lp, ent, ti, tl = (t.cpu() for t in sv.token_logprobs(z.cuda(), tok.cuda(), 4, temperature=T))
    l, e, i, t = R.logprobs(z, tok, 4, T)
    assert ((lp.double() - l).abs() <= 2.0 ** -18 + 2.0 ** -22 * l.abs()).all()
    assert ((ent.double() - e).abs() <= 2.0 ** -18 * (1 + e + math.log(V))).all()
    assert torch.equal(ti.long(), i)
    assert ((tl.double() - t).abs() <= 2.0 ** -18 + 2.0 ** -22 * t.abs()).all()


def test_the_packages_workspaces(sv):
    """A Workspace serves the log-probability and attention calls as it does the verification calls,
    in turn with them, grows with them, and its error word tells what went wrong."""
    g = torch.Generator(device="cuda").manual_seed(2)
    ws = sv.Workspace()
    z = torch.randn((9, 50257), generator=g, device="cuda") * 3
    tok = torch.randint(0, 50257, (9,), generator=g, device="cuda").to(torch.int32)
    cache = sv.KVCache(*R.make_cache_on_gpu(3, 2, 3000, 16, 2, 128))
    q = torch.randn((2, 9, 8, 128), generator=g, device="cuda").to(torch.bfloat16)
    ctx = torch.tensor([2900, 40], dtype=torch.int32, device="cuda")
    draft = tok.view(3, 3)[:, :2].contiguous()
    calls = [lambda **k: sv.token_logprobs(z, tok, 3, **k), lambda **k: sv.paged_attention(q, cache, ctx, lse=True, **k),
             lambda **k: sv.verify_greedy(z.view(3, 3, -1), draft, **k), lambda **k: sv.token_logprobs(z[:1], tok[:1], 0, **k)]
    want = [f() for f in calls]
    for _ in range(3):
        for f, w in zip(calls, want):
            assert all(a is b is None or torch.equal(a, b) for a, b in zip(f(workspace=ws), w))
            assert ws.read_error() == 0
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    other = sv.Workspace()
    got = [f(workspace=other, stream=side) for f in calls]
    torch.cuda.synchronize()
    for r, w in zip(got, want):
        assert all(a is b is None or torch.equal(a, b) for a, b in zip(r, w))
    tok[4] = -1
    z[7] = -math.inf
    lp, *_ = calls[0](workspace=ws)
    assert torch.isnan(lp[[4, 7]]).all()
    calls[1](workspace=ws)                                     # leaves the error word alone
    assert ws.read_error() == sv.SPEC_DEVERR_TOKEN_RANGE | sv.SPEC_DEVERR_EMPTY_ROW
    for bad in (torch.zeros(64, device="cuda"), "ws", 7):
        with pytest.raises(TypeError):
            calls[0](workspace=bad)
        with pytest.raises(TypeError):
            calls[1](workspace=bad)
    with pytest.raises(ValueError):
        sv.token_logprobs(z, tok, 9, workspace=ws)
    with pytest.raises(ValueError):
        sv.paged_attention(q[:, :, :7].contiguous(), cache, ctx, workspace=ws)

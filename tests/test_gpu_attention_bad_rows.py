"""Rows past a sequence's new positions, where something else of the sequence is bad: a page that is
none, a malformed tree, bad lengths.  What they get does not depend on how the work was split."""
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


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("N,G,D", [(4, 2, 128), (4, 2, 64), (12, 2, 256), (12, 4, 128), (40, 4, 128)])
@pytest.mark.parametrize("fault", ["page", "tree"])
@pytest.mark.parametrize("ctx", [[90, 60], [9000, 60], [60, 9000]])    # whole; the bad one split; the bad one whole
def test_rows_past_the_new_positions_are_empty(sv, fp8, N, G, D, fault, ctx):
    g = torch.Generator().manual_seed(N)
    parts = R.make_cache(50, 2, max(ctx) + N, 16, 1, D, fp8)
    q = (torch.randn((2, N, G, D), generator=g)).to(torch.bfloat16)
    par = torch.tensor([[-1] + [n // 2 for n in range(N - 1)]] * 2, dtype=torch.int32)
    new = torch.tensor([N - 2, N - 1], dtype=torch.int32)
    c = torch.tensor(ctx, dtype=torch.int32)
    table = parts[2].clone()
    cache = R.on_gpu(sv, parts)
    want, wl = sv.paged_attention(q.cuda(), cache, c.cuda(), parents=par.cuda(), new_lens=new.cuda(), lse=True)
    if fault == "page":
        table[0, 1] = 1 << 25
    else:
        par[0, 1] = 1
    cache = R.on_gpu(sv, (parts[0], parts[1], table, parts[3], parts[4]))
    out, lse = sv.paged_attention(q.cuda(), cache, c.cuda(), parents=par.cuda(), new_lens=new.cuda(), lse=True)
    assert cache.read_error() == (sv.SPEC_DEVERR_CACHE_RANGE if fault == "page" else sv.SPEC_DEVERR_TREE_PARENT)
    assert torch.isnan(out[0, :N - 2]).all() and torch.isnan(lse[0, :N - 2]).all()
    assert (out[0, N - 2:] == 0).all() and (lse[0, N - 2:] == -math.inf).all()
    assert torch.equal(out[1], want[1]) and torch.equal(lse[1], wl[1])


@pytest.mark.parametrize("N,G", [(4, 2), (12, 4)])
def test_bad_lengths_leave_no_row(sv, N, G):
    parts = R.make_cache(51, 3, 400, 16, 1, 128)
    q = torch.randn((3, N, G, 128)).to(torch.bfloat16)
    c = torch.tensor([300, -1, 200], dtype=torch.int32)
    new = torch.tensor([N - 1, 2, N + 1], dtype=torch.int32)
    cache = R.on_gpu(sv, parts)
    out, lse = sv.paged_attention(q.cuda(), cache, c.cuda(), new_lens=new.cuda(), lse=True)
    assert cache.read_error() == sv.SPEC_DEVERR_CACHE_RANGE
    assert torch.isnan(out[1:]).all() and torch.isnan(lse[1:]).all()
    assert torch.isfinite(out[0]).all() and (out[0, N - 1:] == 0).all()

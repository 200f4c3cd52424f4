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

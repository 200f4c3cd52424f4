"""Products whose tiles are dealt in equal shares, their parts joined through the workspace: tiles of 64 and of 256 weight
rows, in two, three, four and five parts.  The results, and the calls that lean on what CTAs leave one
another there: any contents of a workspace, other operators' among them, replays, waits that run out, a busy memory."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import linear_ref as R  # noqa: E402
import test_gpu_linear_calls as calls  # noqa: E402
from test_gpu_linear_calls import sv  # noqa: E402,F401
from test_linear_plan_cpu import SHARED, SHARES, WAYS  # noqa: E402

SIZES = [s for v in SHARED.values() for s in v]


@pytest.mark.parametrize("want,sizes", [(k, s) for k, v in WAYS.items() for s in v] +
                         [((SHARES, k[0], 2, k[1]), s) for k, v in SHARED.items() for s in v])
def test_way_on_this_device(sv, want, sizes):  # noqa: F811
    way, W, together, _, parts = sv.matmul_plan(*sizes)
    if torch.cuda.get_device_properties(0).multi_processor_count == 152:
        assert (way, W, together, parts) == want


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_result(sv, M, N, K, dtype):  # noqa: F811
    p = R.problem(M + N + K, M, N, K)
    ref, mags = R.matmul(*p)
    first = sv.matmul_e4m3(*p, dtype=dtype)
    assert ((first.double() - ref).abs() <= R.matmul_bound(ref, mags, K, dtype)).all()
    wide = torch.full((M, N + 3), -7.0, dtype=dtype, device="cuda")
    got = sv.matmul_e4m3(*p, dtype=dtype, out=wide[:, 1:N + 1])
    assert torch.equal(got, first) and (wide[:, 0] == -7).all() and (wide[:, N + 1:] == -7).all()


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("check", [calls.test_workspaces_of_any_contents, calls.test_inputs_written_by_the_kernel_before,
                                   calls.test_captured_products, calls.test_wait_limit_zero_times_out_then_recovers])
def test_calls(sv, check, M, N, K):  # noqa: F811
    check(sv, M, N, K)


def test_one_workspace_for_calls_of_all_kinds(sv):  # noqa: F811
    """The words of tickets and parts written over by other operators, and by products of other tiles."""
    w = sv.Workspace()
    g = torch.Generator(device="cuda").manual_seed(0)
    z = torch.randn((64, 50257), generator=g, device="cuda")
    tok = torch.zeros(64, dtype=torch.int32, device="cuda")
    lp = [t.clone() for t in sv.token_logprobs(z, tok, 4)]
    for M, N, K in SIZES:
        p = R.problem(M, M, N, K)
        want = sv.matmul_e4m3(*p, dtype=torch.float32)
        for _ in range(3):
            assert torch.equal(want, sv.matmul_e4m3(*p, dtype=torch.float32, workspace=w))
            assert all(torch.equal(a, b) for a, b in zip(lp, sv.token_logprobs(z, tok, 4, workspace=w)))
    assert w.read_error() == 0


@pytest.mark.parametrize("M,N,K", SIZES)
def test_agrees_with_itself_while_the_memory_is_busy(sv, M, N, K):  # noqa: F811
    p = R.problem(M, M, N, K)
    first = sv.matmul_e4m3(*p, dtype=torch.float32)
    other = torch.empty(32 << 20, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(150):
        if i % 3 == 0:
            other.fill_(i)
        if i % 3 == 1:
            with torch.cuda.stream(side):
                other.add_(1)
        differ += (sv.matmul_e4m3(*p, dtype=torch.float32) != first).sum()
    torch.cuda.synchronize()
    assert int(differ) == 0

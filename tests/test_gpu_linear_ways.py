"""Every way in which a product of more than 64 rows is divided (whole tiles of pairs and of single CTAs in each
width, clusters of two, four and eight CTAs, equal shares with their parts), by sizes that take it: the
result, and the calls that lean on what CTAs tell one another."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import linear_ref as R  # noqa: E402
import test_gpu_linear_calls as calls  # noqa: E402
from test_gpu_linear_calls import sv  # noqa: E402,F401

SHAPES = [
    # pairs: tiles of 64, 128, 192, 256; clusters of two pairs and of four, of two with tiles of 128; shares of
    # tiles of 64 and of 256
    (100, 300, 400), (500, 3000, 400), (600, 4000, 528), (700, 5000, 528), (128, 128, 2064), (128, 70, 8208), (250, 4000, 12304), (700, 1000, 16400),
    (600, 2000, 16400), (2000, 3000, 8192),
    # single CTAs: tiles of 64, 128, 192, 256; clusters of two, four and eight
    (300, 3000, 1040), (257, 5000, 1040), (600, 5000, 528), (300, 12000, 528), (65, 3000, 2064), (100, 2000, 8208), (128, 64, 12304)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_result(sv, M, N, K, dtype):  # noqa: F811
    x, xs, w, ws = R.problem(M + N + K, M, N, K)
    ref, mags = R.matmul(x, xs, w, ws)
    bound = R.matmul_bound(ref, mags, K, dtype)
    first = sv.matmul_e4m3(x, xs, w, ws, dtype=dtype)
    assert ((first.double() - ref).abs() <= bound).all()
    # into rows that are not aligned, and wider than the result
    wide = torch.full((M, N + 3), -7.0, dtype=dtype, device="cuda")
    got = sv.matmul_e4m3(x, xs, w, ws, dtype=dtype, out=wide[:, 1:N + 1])
    assert torch.equal(got, first) and (wide[:, 0] == -7).all() and (wide[:, N + 1:] == -7).all()
    for _ in range(30):
        assert torch.equal(sv.matmul_e4m3(x, xs, w, ws, dtype=dtype), first)


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("check", [calls.test_workspaces_of_any_contents, calls.test_inputs_written_by_the_kernel_before,
                                   calls.test_captured_products, calls.test_wait_limit_zero_times_out_then_recovers])
def test_calls(sv, check, M, N, K):  # noqa: F811
    check(sv, M, N, K)

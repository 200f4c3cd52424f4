"""Products of some of the rows that a call has rounded: one row, or more than 64, from anywhere, their scales where that
call left them, and a single row's scales in every order; the same numbers as with the scales laid out anew."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import linear_ref as R  # noqa: E402
from test_gpu_linear_calls import sv  # noqa: E402,F401


def anew(scale):
    """The same scales as a quantising call lays them out, NaN between them."""
    rows, blocks = scale.shape
    t = torch.full((blocks, -(-rows // 4) * 4), float("nan"), device="cuda")
    t[:, :rows] = scale.t()
    return t[:, :rows].t()


def check(sv, x, xs, w, ws, dtype=torch.float32):  # noqa: F811
    got = sv.matmul_e4m3(x, xs, w, ws, dtype=dtype)
    ref, mags = R.matmul(x, xs, w, ws)
    assert ((got.double() - ref).abs() <= R.matmul_bound(ref, mags, x.shape[1], dtype)).all()
    assert torch.equal(got, sv.matmul_e4m3(x, anew(xs), w, ws, dtype=dtype))
    return got


@pytest.mark.parametrize("rows", [2, 5, 6, 7, 8, 131])
@pytest.mark.parametrize("N,K", [(1000, 4096), (200, 144), (300, 16), (128, 12304), (6144, 4096)])
def test_last_row(sv, rows, N, K):  # noqa: F811
    g = torch.Generator(device="cuda").manual_seed(rows + N)
    q, s = sv.quantize_e4m3(torch.randn((rows, K), generator=g, device="cuda"))
    _, _, w, ws = R.problem(N, 1, N, K)
    check(sv, q[-1:], s[-1:], w, ws)
    check(sv, q[1:2], s[1:2], w, ws, torch.bfloat16)
    for i in (0, rows - 1):                                   # without the leading dimension
        one = sv.matmul_e4m3(q[i], s[i], w, ws)
        assert one.shape == (N,) and torch.equal(one, sv.matmul_e4m3(q[i:i + 1], s[i:i + 1], w, ws)[0])


@pytest.mark.parametrize("K", [128, 400, 4096, 30000, 40960])
@pytest.mark.parametrize("stride", [1, 3, 4, 9])
@pytest.mark.parametrize("at", [0, 1, 2])
def test_one_rows_scales_in_any_order(sv, K, stride, at):  # noqa: F811
    blocks = -(-K // 128)
    x, xs, w, ws = R.problem(K, 1, 300, K)
    store = torch.full((blocks * stride + 4,), float("nan"), device="cuda")
    scale = store[at:].as_strided((1, blocks), (blocks * stride, stride), at)
    scale.copy_(xs)
    check(sv, x, scale, w, ws)


@pytest.mark.parametrize("M", [65, 66, 127, 300, 700])
@pytest.mark.parametrize("at,more", [(1, 0), (2, 3), (3, 1), (4, 2)])
def test_many_rows_from_anywhere(sv, M, at, more):  # noqa: F811
    K, N = 1040, 700
    x, xs, w, ws = R.problem(M + at, M, N, K)
    store = torch.full((9, at + M + more), float("nan"), device="cuda")
    store[:, at:at + M] = xs.t()
    rows = torch.full((M + at, K), 0x7f, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    rows.view(torch.uint8)[at:] = x.view(torch.uint8)
    check(sv, rows[at:], store[:, at:at + M].t(), w, ws)


def test_captured_and_on_rewritten_scales(sv):  # noqa: F811
    """A single row's loads see what the kernel before has written, captured ones too."""
    K, N = 4096, 1000
    sets = [R.problem(i, 1, N, K) for i in range(3)]
    want = [sv.matmul_e4m3(*p, dtype=torch.float32) for p in sets]
    x, _, w, ws = (t.clone() for t in sets[0])
    scale = torch.zeros(33, device="cuda")[1:].view(1, 32)
    graph = torch.cuda.CUDAGraph()
    sv.matmul_e4m3(x, scale, w, ws)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        held = sv.matmul_e4m3(x, scale, w, ws, dtype=torch.float32)
    for turn in range(9):
        p = sets[turn % 3]
        x.view(torch.uint8).copy_(p[0].view(torch.uint8))
        w.view(torch.uint8).copy_(p[2].view(torch.uint8))
        ws.copy_(p[3])
        scale.copy_(p[1])
        assert torch.equal(sv.matmul_e4m3(x, scale, w, ws, dtype=torch.float32), want[turn % 3])
        graph.replay()
        assert torch.equal(held, want[turn % 3])


def test_waits_that_run_out(sv):  # noqa: F811
    x, _, w, ws = R.problem(1, 1, 1000, 4096)
    scale = torch.ones(33, device="cuda")[1:].view(1, 32)
    want = sv.matmul_e4m3(x, scale, w, ws)
    mine = sv.Workspace()
    sv.spec_verify_set_wait_limit(0)
    try:
        bad = sv.matmul_e4m3(x, scale, w, ws, workspace=mine)
        torch.cuda.synchronize()
    finally:
        sv.spec_verify_set_wait_limit(sv.spec_verify_default_wait_limit())
    assert mine.read_error() == sv.SPEC_DEVERR_TIMEOUT and bad.isnan().all()
    assert torch.equal(want, sv.matmul_e4m3(x, scale, w, ws, workspace=mine)) and mine.read_error() == 0


@pytest.mark.parametrize("M", [2, 3, 16, 64])
def test_refused(sv, M):  # noqa: F811
    x, xs, w, ws = R.problem(M, M, 64, 256)
    store = torch.zeros((2, 68), device="cuda")
    with pytest.raises(sv.SpecVerifyError):
        sv.matmul_e4m3(x, store[:, 1:M + 1].t(), w, ws)
    assert sv.matmul_e4m3(x, store[:, 4:M + 4].t(), w, ws).shape == (M, 64)

"""Sums of a product are fp32, those in tensor memory too: what 24 bits hold is exact, whichever way it is divided."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_linear_calls import sv  # noqa: E402,F401
from test_linear_plan_cpu import SHARED, WAYS  # noqa: E402


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def unit(rows, cols):
    return torch.ones((cols, -(-rows // 4) * 4), device="cuda")[:, :rows].t()


@pytest.mark.parametrize("M,N,K", [(1, 300, 4096), (16, 300, 4096), (20, 1000, 400), (64, 1000, 12304), (64, 130, 208)] +
                         [s for v in (*WAYS.values(), *SHARED.values()) for s in v[:1]])
def test_sums_that_24_bits_hold(sv, M, N, K):  # noqa: F811
    """Whole numbers up to 8 with scales that are powers of two: every sum of every part is a whole number under
    64 K < 2^22 times one power of two."""
    g = gen(M + N + K)
    x, w = (torch.randint(-8, 9, s, generator=g, device="cuda").float().to(torch.float8_e4m3fn) for s in ((M, K), (N, K)))
    blocks = -(-K // 128)
    got = sv.matmul_e4m3(x, unit(M, blocks) * 0.25, w, torch.full((-(-N // 128), blocks), 2.0, device="cuda"), dtype=torch.float32)
    ref = (x.double() @ w.double().t()) / 2
    assert torch.equal(got.double(), ref)
    half = sv.matmul_e4m3(x, unit(M, blocks) * 0.25, w, torch.full((-(-N // 128), blocks), 2.0, device="cuda"))
    assert torch.equal(half, ref.float().to(torch.bfloat16))


@pytest.mark.parametrize("M", [5, 40, 64, 120, 140, 600])
@pytest.mark.parametrize("at", [0, 5, 40, 127])
def test_small_products_beside_a_large_one(sv, M, at):  # noqa: F811
    """448 * 64 and 127 products of 2^-6: multiples of 2^-6 under 2^15, 21 bits."""
    x = torch.full((M, 128), 1.0, device="cuda").to(torch.float8_e4m3fn)
    w = torch.full((128, 128), 2.0 ** -6, device="cuda").to(torch.float8_e4m3fn)
    w[:, at], x[:, at] = 448.0, 64.0
    got = sv.matmul_e4m3(x, unit(M, 1), w, torch.ones((1, 1), device="cuda"), dtype=torch.float32)
    assert (got == 448.0 * 64 + 127 / 64).all()

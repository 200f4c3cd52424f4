"""8-bit outputs are the nearest values, but for what the fp32 arithmetic before the rounding moves."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import linear_ref as R  # noqa: E402
from test_gpu_linear_calls import sv  # noqa: E402,F401
from test_linear_nearest_cpu import check_nearest  # noqa: E402

ROWS = [(1, 4096), (7, 64), (33, 1008), (129, 2048), (1152, 4096), (3, 40000)]


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


@pytest.mark.parametrize("rows,dim", ROWS)
@pytest.mark.parametrize("xt", [torch.bfloat16, torch.float32])
def test_norm(sv, rows, dim, xt):  # noqa: F811
    g = gen(rows + dim)
    x = torch.randn((rows, dim), generator=g, device="cuda").to(xt)
    r = (3 * torch.randn((rows, dim), generator=g, device="cuda")).to(torch.bfloat16)
    w = (torch.rand(dim, generator=g, device="cuda") + 0.5).to(torch.bfloat16)
    # the row's factor falls out of y / t: h, h w and the factor 448 / t twice over, a rounding of 2^-24 each: 6
    check_nearest(sv.add_norm(x, w, r, e4m3=True)[0], R.norm(x, w, r, 1e-6)[0], 2.0 ** -21)
    check_nearest(sv.add_norm(x, e4m3=True)[0], R.norm(x, None, None, 1e-6)[0], 2.0 ** -21)


@pytest.mark.parametrize("rows,dim", ROWS)
@pytest.mark.parametrize("kind,slack", [("silu", 2.0 ** -17), ("gelu", 2.0 ** -15)])
def test_activation(sv, rows, dim, kind, slack):  # noqa: F811
    """e^-s is off by 2 steps of 2^-23 and s times what s is off by: of silu (|s| = 1.44 |gate| <= 30) two roundings, of
    gelu five, where |s| <= 60 (beyond, what is left of the gate is under 2^-55).  Sum, reciprocal and products are 5 halves of a
    step more, t is off by as much again and the last product by two roundings: 30 0.7 2 + 9 = 51 times two and 2 of 2^-24
    for silu, 60 0.7 5 + 9 = 219 times two and 2 for gelu."""
    x = (3 * torch.randn((rows, 2 * dim), generator=gen(rows + dim), device="cuda")).to(torch.bfloat16)
    check_nearest(sv.gated_act(x, act=kind, e4m3=True)[0], R.act(*x.chunk(2, -1), kind), slack)


@pytest.mark.parametrize("rows,dim", ROWS)
@pytest.mark.parametrize("high", [1, 128])
def test_rounding(sv, rows, dim, high):  # noqa: F811
    x = torch.randn((rows, dim), generator=gen(rows + dim), device="cuda")
    for t in (x, x.to(torch.bfloat16)):
        check_nearest(sv.quantize_e4m3(t, block_rows=high)[0], t.double(), 2.0 ** -23, high)       # 448 / t, the product

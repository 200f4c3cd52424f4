"""Rounding to e4m3 checked for the nearest value, with what the fp32 arithmetic before may move; that the check sees a
rounding towards zero, and a value that is one step off."""
import pytest

torch = pytest.importorskip("torch")

import linear_ref as R  # noqa: E402


def nearest_e4m3(v):
    """The nearest e4m3 values (ties to even, saturating) of v in 64 bits."""
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp(-6, 8) - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def check_nearest(q, y, slack, high=1):
    """q = e4m3(v (1 + d)), v = y 448 / t in 64 bits and |d| <= slack: then |q - v (1 + d)| is at most that of the value nearest to
    v, and so |q - v| at most |nearest - v| + 2 |v| slack.  (And 2^-30 for what is nothing beside its block.)"""
    rows, dim = y.shape
    top = R.block_top(y, high).clamp_min(1e-20).repeat_interleave(high, 0)[:rows].repeat_interleave(R.BLOCK, 1)[:, :dim]
    v = y * 448 / top
    off, least = (q.double() - v).abs(), (nearest_e4m3(v) - v).abs()
    bad = off > least + 2 * v.abs() * slack + 2.0 ** -30
    assert not bad.any(), (int(bad.sum()), v[bad][:8].tolist(), q.double()[bad][:8].tolist())


def test_nearest_is_torchs_rounding():
    g = torch.Generator().manual_seed(0)
    v = torch.randn((64, 512), generator=g) * torch.exp2(torch.randint(-14, 9, (64, 512), generator=g).float())
    v = torch.cat([v.flatten(), torch.tensor([0.0, -0.0, 448.0, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, 464.0, 17.0, 19.0, 1.0625])]).clamp(-448, 448)
    assert torch.equal(nearest_e4m3(v.double()), v.to(torch.float8_e4m3fn).double())


def test_the_check_sees_wrong_neighbours():
    y = torch.randn((8, 512), generator=torch.Generator().manual_seed(1), dtype=torch.float64)
    v = y * 448 / R.block_top(y).repeat_interleave(R.BLOCK, 1)
    q = nearest_e4m3(v)
    check_nearest(q, y, 2.0 ** -30)
    moved = v * (1 + 2.0 ** -18)
    check_nearest(nearest_e4m3(moved), y, 2.0 ** -18)
    _, e = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), (e - 1).clamp(-6, 8) - 3)
    with pytest.raises(AssertionError):
        check_nearest(torch.trunc(v / step) * step, y, 2.0 ** -17)
    one = q.clone()
    one[3, 77] += step[3, 77]
    with pytest.raises(AssertionError):
        check_nearest(one, y, 2.0 ** -17)

"""The target model's dense side in 64 bits: norm, gated activation, rounding to e4m3 with a scale for each
block of 128, and the product of scaled 8-bit matrices.  Plain forms for the tests."""
import torch

BLOCK = 128


def value(q, scale, high=1):
    """What e4m3 values q [rows, dim] stand for, scale [rows / high, blocks]."""
    rows, dim = q.shape
    s = scale.double().repeat_interleave(high, 0)[:rows].repeat_interleave(BLOCK, 1)[:, :dim]
    return q.double() * s


def block_top(y, high=1):
    """The largest magnitude of each block, [rows / high, blocks]."""
    rows, dim = y.shape
    p = torch.nn.functional.pad(y.abs(), (0, -dim % BLOCK, 0, -rows % high))
    return p.view(p.shape[0] // high, high, -1, BLOCK).amax((1, 3))


def check_e4m3(q, scale, y, high=1, slack=2.0 ** -20):
    """q and scale against rows y in 64 bits of which the fp32 arithmetic before is off by `slack` of a
    value at most (or of the block's largest, for what cancels)."""
    rows, dim = y.shape
    top = block_top(y, high).clamp_min(1e-20)
    assert q.shape == y.shape and scale.shape == top.shape
    assert ((scale.double() - top / 448).abs() <= top / 448 * (slack + 2.0 ** -23)).all()
    big = top.repeat_interleave(high, 0)[:rows].repeat_interleave(BLOCK, 1)[:, :dim]
    # half a step of a value is 2^-4 of it, half of the least step 2^-10 of 2^0
    bound = y.abs() * 2.0 ** -4 + big / 448 * 2.0 ** -10 + big * (slack + 2.0 ** -22)
    err = (value(q, scale, high) - y).abs()
    assert (err <= bound).all(), (err / bound).max()
    # and the nearest value nearly always: the rounding errors of a uniform value have 1 / 3 of half a step rms
    assert q.float().abs().max() <= 448


def norm(x, weight, residual, eps):
    h = x.double() if residual is None else x.double() + residual.double()
    y = h / torch.sqrt(h.square().mean(-1, keepdim=True) + eps)
    return (y if weight is None else y * weight.double()), h


def act(gate, up, kind):
    g = gate.double()
    if kind == "silu":
        return g * torch.sigmoid(g) * up.double()
    return 0.5 * g * (1 + torch.tanh((2 / torch.pi) ** 0.5 * (g + 0.044715 * g ** 3))) * up.double()


def matmul(x, xs, w, ws):
    """(the product, the product of the magnitudes) in 64 bits."""
    a, b = value(x, xs), value(w, ws, BLOCK)
    return a @ b.t(), a.abs() @ b.abs().t()


def matmul_bound(ref, mags, K, dtype):
    """How far a product may be off: a block's 128 sums, each off by at most a step of fp32 (2^-23) of what the
    magnitudes add up to, then three roundings a block (the scales' product, its product, the sum) over
    K / 128 blocks and up to 8 parts, and half a step of the output."""
    blocks = -(-K // BLOCK)
    return mags * (128 * 2.0 ** -23 + (2 + blocks + 8) * 2.0 ** -24) + ref.abs() * (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24)


def rand_e4m3(g, rows, cols):
    t = torch.randn((rows, cols), generator=g, device=g.device) * 110
    return t.clamp_(-448, 448).to(torch.float8_e4m3fn)


def scales(g, rows, blocks):
    """[rows, blocks] with the scales of a block side by side; what lies between is NaN."""
    t = torch.full((blocks, -(-rows // 4) * 4), float("nan"), device=g.device)
    t[:, :rows] = torch.rand((blocks, rows), generator=g, device=g.device) + 0.5
    return t[:, :rows].t()


def problem(seed, M, N, K, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    blocks = -(-K // BLOCK)
    ws = (torch.rand((-(-N // BLOCK), blocks), generator=g, device=device) + 0.5) / (110 * 110 * K ** 0.5)
    return rand_e4m3(g, M, K), scales(g, M, blocks), rand_e4m3(g, N, K), ws

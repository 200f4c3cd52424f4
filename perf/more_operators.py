"""The target model's dense side of a verification step, as measurable cases.

Between the cache and attention calls a target model normalises its hidden rows and
multiplies them with its weights.  With weights and rows held in 8 bits that takes four
operators: the residual's addition with the root-mean-square norm (`add_norm`), the gated
activation between the two products of a feed-forward part (`gated_act`), both with an
output in 8 bits, the rounding of rows and weights to 8 bits (`quantize_e4m3`), and the
product of two 8-bit matrices (`matmul_e4m3`).  Rows carry a scale for each 128 of their
elements, weights one for each 128 x 128.

`run` computes each of them in its plain form (elementary torch operations in 32 bits,
rounded once at the end) or, where `own` is true, through this package.
"""
import math

import torch

own = False

BLOCK = 128              # elements that share a scale
FP8_MAX = 448.0          # largest finite e4m3 value
FP8_AMAX_FLOOR = 1e-20   # blocks below this quantise with its scale (and so to zero)
EPS = 1e-6


def _sv():
    import speculative_decoding_verification_59_gb300 as sv
    return sv


# ---- the cases ------------------------------------------------------------------------
def listed():
    return [
        # The hidden row of one new token before its query, key and value projection.
        dict(name="norm-one", op="norm", rows=1, dim=4096, xf32=False, rf32=False, add=True, fp8=True),
        # A prompt of 8192 tokens with the residual kept in 32 bits, on to a product in bf16.
        dict(name="norm-prompt", op="norm", rows=8192, dim=4096, xf32=False, rf32=True, add=True, fp8=False),
        # One chain of 7 positions between the feed-forward products.
        dict(name="act-one", op="act", rows=7, dim=12288, act="silu", fp8=True),
        # 32 draft trees of 36 nodes there.
        dict(name="act-trees", op="act", rows=1152, dim=12288, act="silu", fp8=True),
        # The attention's output of the same trees, for the output projection.
        dict(name="quantize-trees", op="quantize", rows=1152, dim=4096, xf32=False, block=1),
        # The gate and up weights of a feed-forward part, when a model is loaded.
        dict(name="quantize-weights", op="quantize", rows=24576, dim=4096, xf32=False, block=128),
        # Query, key and value projection of one new token (32 and 2 x 8 heads of 128): latency.
        dict(name="matmul-one", op="matmul", M=1, N=6144, K=4096, f32=False),
        # Down projection of one sequence's 8 positions: few tiles, a long contraction.
        dict(name="matmul-chain", op="matmul", M=8, N=4096, K=12288, f32=False),
        # Logits of a small model with a vocabulary of 1000, odd sizes throughout.
        dict(name="matmul-odd", op="matmul", M=77, N=1000, K=1040, f32=True),
        # Gate and up projection of the ordinary step: 64 sequences of 8 positions.
        dict(name="matmul-b64", op="matmul", M=512, N=24576, K=4096, f32=False),
        # Down projection of 32 draft trees of 36 nodes.
        dict(name="matmul-trees", op="matmul", M=1152, N=4096, K=12288, f32=False),
        # Logits of all 512 positions of 64 chains over a vocabulary of 151936.
        dict(name="matmul-head", op="matmul", M=512, N=151936, K=4096, f32=False),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["norm", "act", "quantize", "matmul", "matmul", "matmul"])
    dim = 16 * _logint(rng, 4, 1024)
    if op == "norm":
        return dict(op=op, rows=_logint(rng, 1, max(1, int(3e7 / dim))), dim=dim, xf32=rng.random() < 0.3, rf32=rng.random() < 0.4, add=rng.random() < 0.8,
                    fp8=rng.random() < 0.6)
    if op == "act":
        return dict(op=op, rows=_logint(rng, 1, max(1, int(1.2e7 / dim))), dim=dim, act=rng.choice(["silu", "gelu"]), fp8=rng.random() < 0.7)
    if op == "quantize":
        return dict(op=op, rows=_logint(rng, 1, max(1, int(5e7 / dim))), dim=dim, xf32=rng.random() < 0.3, block=rng.choice([1, 1, 128]))
    M, N = _logint(rng, 1, 2048), _logint(rng, 64, 40000)
    K = 16 * _logint(rng, 8, max(8, min(1024, int(1.2e11 / M / N / 16), int(6e8 / N / 16))))
    return dict(op=op, M=M, N=N if rng.random() < 0.5 else (N + 127) // 128 * 128, K=K, f32=rng.random() < 0.3)


# ---- inputs ---------------------------------------------------------------------------
def _randn(g, dev, shape, dtype, spread=1.0):
    return (torch.randn(shape, generator=g, device=dev) * spread).to(dtype)


def _rand8(g, dev, rows, cols):
    """8-bit contents over the whole e4m3 range, of deviation 110."""
    t = torch.empty((rows, cols), device=dev, dtype=torch.float8_e4m3fn)
    step = max(1, (1 << 25) // cols)
    for lo in range(0, rows, step):
        part = torch.randn((min(step, rows - lo), cols), generator=g, device=dev)
        t[lo:lo + step] = part.mul_(110).clamp_(-FP8_MAX, FP8_MAX).to(torch.float8_e4m3fn)
    return t


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    c = case
    s = {"op": c["op"], "case": c}
    if c["op"] == "matmul":
        M, N, K = c["M"], c["N"], c["K"]
        kb, nb = -(-K // BLOCK), -(-N // BLOCK)
        s["x"], s["w"] = _rand8(g, dev, M, K), _rand8(g, dev, N, K)
        # rows' scales lie one block after the other, as the quantising operators leave them
        s["xs"] = ((torch.rand((kb, (M + 3) // 4 * 4), generator=g, device=dev) + 0.5) / 110)[:, :M].t()
        s["ws"] = (torch.rand((nb, kb), generator=g, device=dev) + 0.5) / (110 * math.sqrt(K))
        return s
    rows, dim = c["rows"], c["dim"]
    xt = torch.float32 if c.get("xf32") else torch.bfloat16
    if c["op"] == "norm":
        s["x"] = _randn(g, dev, (rows, dim), xt)
        # a residual has a few channels far larger than the others
        loud = torch.ones(dim, device=dev)
        loud[torch.randint(0, dim, (max(1, dim // 512),), generator=g, device=dev)] = 30.0
        s["r"] = _randn(g, dev, (rows, dim), torch.float32 if c["rf32"] else torch.bfloat16, 4 * loud) if c["add"] else None
        s["w"] = (torch.rand(dim, generator=g, device=dev) + 0.5).to(torch.bfloat16)
    elif c["op"] == "act":
        s["x"] = _randn(g, dev, (rows, 2 * dim), xt, 2.0)        # gate and up side by side
    else:
        s["x"] = _randn(g, dev, (rows, dim), xt, 0.02 if c["block"] > 1 else 1.0)
    return s


# ---- the plain forms ------------------------------------------------------------------
def _blocks(x):
    """x [rows, dim] as [rows, blocks, 128], zeros behind the last element."""
    rows, dim = x.shape
    pad = -dim % BLOCK
    return torch.nn.functional.pad(x, (0, pad)).view(rows, -1, BLOCK)


def _quantise(y, high):
    """y [rows, dim] in 32 bits to e4m3 with a scale for each `high` x 128 of its elements."""
    rows, dim = y.shape
    if high > 1:
        t = _blocks(torch.nn.functional.pad(y, (0, 0, 0, -rows % high)))
        amax = t.view(-1, high, t.shape[1], BLOCK).abs().amax((1, 3)).clamp_min(FP8_AMAX_FLOOR)
        times = (FP8_MAX / amax).repeat_interleave(high, 0)[:rows]
    else:
        amax = _blocks(y).abs().amax(-1).clamp_min(FP8_AMAX_FLOOR)
        times = FP8_MAX / amax
    q = (_blocks(y) * times[..., None]).view(rows, -1)[:, :dim]
    return {"q": q.to(torch.float8_e4m3fn), "scale": amax / FP8_MAX}


def _out(y, fp8):
    return _quantise(y, 1) if fp8 else {"y": y.to(torch.bfloat16)}


def _plain_norm(s):
    h = s["x"].to(torch.float32)
    if s["r"] is not None:
        h = h + s["r"].to(torch.float32)
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["w"].to(torch.float32)
    out = _out(y, s["case"]["fp8"])
    if s["r"] is not None:
        out["sum"] = h.to(s["r"].dtype)
    return out


def _plain_act(s):
    gate, up = s["x"].to(torch.float32).chunk(2, -1)
    if s["case"]["act"] == "silu":
        y = gate / (1 + torch.exp(-gate)) * up
    else:
        y = 0.5 * gate * (1 + torch.tanh(math.sqrt(2 / math.pi) * (gate + 0.044715 * gate * gate * gate))) * up
    return _out(y, s["case"]["fp8"])


def _plain_matmul(s):
    M, N, K = s["case"]["M"], s["case"]["N"], s["case"]["K"]
    x = (_blocks(s["x"].to(torch.float32)) * s["xs"][..., None]).view(M, -1)[:, :K]
    w = (_blocks(s["w"].to(torch.float32)) * s["ws"].repeat_interleave(BLOCK, 0)[:N, :, None]).view(N, -1)[:, :K]
    return {"out": (x @ w.t()).to(torch.float32 if s["case"]["f32"] else torch.bfloat16)}


def _own(s):
    sv, c = _sv(), s["case"]
    if s["op"] == "norm":
        got = sv.add_norm(s["x"], s["w"], s["r"], eps=EPS, e4m3=c["fp8"])
        got = got if isinstance(got, tuple) else (got,)
        return dict(zip(("q", "scale", "sum") if c["fp8"] else ("y", "sum"), got))
    if s["op"] == "act":
        got = sv.gated_act(s["x"], act=c["act"], e4m3=c["fp8"])
        return {"q": got[0], "scale": got[1]} if c["fp8"] else {"y": got}
    if s["op"] == "quantize":
        q, scale = sv.quantize_e4m3(s["x"], block_rows=c["block"])
        return {"q": q, "scale": scale}
    return {"out": sv.matmul_e4m3(s["x"], s["xs"], s["w"], s["ws"], dtype=torch.float32 if c["f32"] else torch.bfloat16)}


def run(state):
    if own:
        return _own(state)
    op = state["op"]
    if op == "norm":
        return _plain_norm(state)
    if op == "act":
        return _plain_act(state)
    if op == "quantize":
        return _quantise(state["x"].to(torch.float32), state["case"]["block"])
    return _plain_matmul(state)


# ---- what a pass cannot do without ----------------------------------------------------
def work(case):
    c = case
    if c["op"] == "matmul":
        M, N, K = c["M"], c["N"], c["K"]
        kb, nb = -(-K // BLOCK), -(-N // BLOCK)
        return {"bytes": M * K + N * K + 4 * kb * (M + nb) + M * N * (4 if c["f32"] else 2), "flops": 2 * M * N * K}
    rows, dim = c["rows"], c["dim"]
    n, blocks = rows * dim, -(-dim // BLOCK)
    out = n + 4 * rows * blocks if c.get("fp8", True) else 2 * n
    if c["op"] == "norm":
        both = 2 * (4 if c["rf32"] else 2) if c["add"] else 0
        return {"bytes": n * ((4 if c["xf32"] else 2) + both) + out + 2 * dim, "flops": 6 * n}
    if c["op"] == "act":
        return {"bytes": 4 * n + out, "flops": 8 * n}
    return {"bytes": n * (4 if c["xf32"] else 2) + n + 4 * -(-rows // c["block"]) * blocks, "flops": 3 * n}


# ---- 64 bits, written apart -----------------------------------------------------------
def _nearest_e4m3(x):
    """The nearest e4m3 value (ties to even), saturating: 3 mantissa bits, least exponent -6."""
    e = torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -30))).clamp(-6, 8)
    step = torch.pow(2.0, e - 3)
    return (torch.round(x / step) * step).clamp(-FP8_MAX, FP8_MAX)


def _exact_e4m3(y, high):
    rows, dim = y.shape
    q = torch.empty_like(y)
    scale = torch.empty((-(-rows // high), -(-dim // BLOCK)), dtype=torch.float64, device=y.device)
    for b in range(scale.shape[1]):
        part = y[:, b * BLOCK:(b + 1) * BLOCK]
        top = part.abs().max(dim=1).values
        if high > 1:
            top = torch.stack([t.max() for t in top.split(high)])
        top = torch.maximum(top, torch.tensor(FP8_AMAX_FLOOR, dtype=torch.float64, device=y.device))
        scale[:, b] = top / FP8_MAX
        wide = top if high == 1 else top[torch.arange(rows, device=y.device) // high]
        q[:, b * BLOCK:(b + 1) * BLOCK] = _nearest_e4m3(part * (FP8_MAX / wide)[:, None])
    return {"q": q, "scale": scale}


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "matmul":
        M, N, K = c["M"], c["N"], c["K"]
        if 2 * M * N * K > 3e12:
            return None
        dev = s["x"].device
        of_k = torch.arange(K, device=dev) // BLOCK
        x = s["x"].to(torch.float64) * s["xs"].to(torch.float64)[:, of_k]
        out = torch.empty((M, N), dtype=torch.float64, device=dev)
        for lo in range(0, N, 8192):
            n = torch.arange(lo, min(lo + 8192, N), device=dev)
            w = s["w"][lo:lo + 8192].to(torch.float64) * s["ws"].to(torch.float64)[n // BLOCK][:, of_k]
            out[:, lo:lo + 8192] = torch.einsum("mk,nk->mn", x, w)
        return {"out": out}
    if c["op"] == "norm":
        h = s["x"].double()
        if c["add"]:
            h = s["r"].double() + h
        y = s["w"].double() * h / torch.sqrt(torch.square(h).sum(-1, keepdim=True) / c["dim"] + EPS)
        out = _exact_e4m3(y, 1) if c["fp8"] else {"y": y}
        return {**out, "sum": h} if c["add"] else out
    if c["op"] == "act":
        gate, up = s["x"][:, :c["dim"]].double(), s["x"][:, c["dim"]:].double()
        if c["act"] == "silu":
            y = gate * torch.sigmoid(gate) * up
        else:
            # (1 + tanh(t)) / 2 is the logistic function of 2 t
            y = gate * torch.sigmoid(2 * math.sqrt(2 / math.pi) * gate * (1 + 0.044715 * gate ** 2)) * up
        return _exact_e4m3(y, 1) if c["fp8"] else {"y": y}
    return _exact_e4m3(s["x"].double(), c["block"])

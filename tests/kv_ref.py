"""Plain 64-bit forms of the cache, attention and log-probability calls, on the CPU, and
random paged caches.  The tolerances that the GPU tests use are derived here."""
import math

import torch

U_BF16 = 2.0 ** -8        # unit roundoff of an 8-bit significand
U_F16 = 2.0 ** -11
U_F32 = 2.0 ** -24
F8 = torch.float8_e4m3fn


def make_cache(seed, B, tokens, page, H, D, fp8=False, hnd=False, layers=None, extra=3, max_pages=None):
    """(k, v, table, k_scale, v_scale) on the CPU: random rows, pages dealt out of order, unused
    table entries -1, rows of unused pages NaN."""
    g = torch.Generator().manual_seed(seed)
    per = -(-tokens // page)
    pages = B * per + extra
    width = per + 2 if max_pages is None else max_pages
    table = torch.full((B, width), -1, dtype=torch.int32)
    perm = torch.randperm(pages, generator=g)
    table[:, :per] = perm[:B * per].view(B, per).to(torch.int32)
    lead = () if layers is None else (layers,)
    shape = (*lead, pages, H, page, D) if hnd else (*lead, pages, page, H, D)
    out = []
    for _ in range(2):
        x = torch.randn(shape, generator=g)
        unused = perm[B * per:]
        x[(slice(None), unused) if layers else unused] = math.nan
        if fp8:
            sc = (torch.rand(shape[:-1], generator=g) + 0.5) / 100
            y = (x / sc[..., None]).clamp(-448, 448).to(F8)
            out.append((y.transpose(-2, -3) if hnd else y, sc.transpose(-1, -2) if hnd else sc))
        else:
            y = x.to(torch.bfloat16)
            out.append((y.transpose(-2, -3) if hnd else y, None))
    (k, ks), (v, vs) = out
    return k, v, table, ks, vs


def make_cache_on_gpu(seed, B, tokens, page, H, D, fp8=False):
    """make_cache for large ones, made on the GPU."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    per = -(-tokens // page)
    pages = B * per + 3
    table = torch.randperm(pages, generator=g, device="cuda")[:B * per].view(B, per).to(torch.int32)
    out = []
    for _ in range(2):
        x = torch.randn((pages, page, H, D), generator=g, device="cuda")
        sc = (torch.rand((pages, page, H), generator=g, device="cuda") + 0.5) / 100 if fp8 else None
        out.append(((x / sc[..., None]).clamp(-448, 448).to(F8) if fp8 else x.to(torch.bfloat16), sc))
    (k, ks), (v, vs) = out
    return k, v, table, ks, vs


def cuda_like(t):
    """A copy on the GPU with t's strides."""
    if t is None:
        return None
    order = sorted(range(t.dim()), key=lambda d: -t.stride(d))
    p = t.permute(order).contiguous().cuda()
    inv = [order.index(d) for d in range(t.dim())]
    return p.permute(inv)


def on_gpu(sv, parts):
    k, v, table, ks, vs = (cuda_like(t) for t in parts)
    return sv.KVCache(k, v, table.contiguous(), ks, vs)


def rows(x, scale, table, b, n):
    """Positions 0..n-1 of sequence b in 64 bits: [n, H, D]."""
    page = x.shape[-3]
    t = torch.arange(n)
    pg = table[b].long()[t // page]
    y = x.float()[pg, t % page].double()
    return y if scale is None else y * scale[pg, t % page].double()[..., None]


def ancestors(parents):
    N = len(parents)
    m = torch.zeros((N, N), dtype=torch.bool)
    for n in range(N):
        a = n
        while a >= 0:
            m[n, a] = True
            a = int(parents[a])
    return m


def attention(q, k, v, table, ks, vs, ctx, nb, parents=None, scale=None):
    """For one sequence after the other: out, lse and their tolerances, [B, N, Hq, D] and
    [B, N, Hq].

    The kernel's scores are fp32 sums of exact products: off by at most (D + 2) u32 sum |q k|
    scale, plus 4 u32 |s| for the scaling and the exponent's argument; call the largest ds.  Its
    probabilities are rounded to bf16 (fp16 for an 8-bit cache) before they meet the values, the
    result to bf16: |error| <= u_bf16 |out| + (u_p + 2 ds + 2^-18) sum p |v|, the last term
    for fp32 sums in any order.  lse: ds + 2^-20 (1 + |lse|)."""
    B, N, Hq, D = q.shape
    H = k.shape[-2]
    G = Hq // H
    scale = D ** -0.5 if scale is None else scale
    outs, lses, tol_o, tol_l = [], [], [], []
    for b in range(B):
        n, c = int(nb[b]), int(ctx[b])
        o = torch.zeros((N, Hq, D), dtype=torch.float64)
        l = torch.full((N, Hq), -math.inf, dtype=torch.float64)
        to, tl = torch.zeros_like(o), torch.zeros_like(l)
        if n > 0:
            K, V = rows(k, ks, table, b, c + n), rows(v, vs, table, b, c + n)
            sees = torch.ones((n, c + n), dtype=torch.bool)
            sees[:, c:] = torch.tril(torch.ones(n, n)).bool() if parents is None else ancestors(parents[b, :n])
            for h in range(Hq):
                # masked entries may hold anything: they are taken out before the products
                for i in range(n):
                    s_ = sees[i]
                    Kh, Vh = K[s_, h // G], V[s_, h // G]
                    x = (Kh @ q[b, i, h].double()) * scale
                    l[i, h] = torch.logsumexp(x, 0)
                    p = torch.softmax(x, 0)
                    o[i, h] = p @ Vh
                    mag = ((Kh.abs() @ q[b, i, h].double().abs()) * abs(scale)).max()
                    ds = (D + 2) * U_F32 * mag + 4 * U_F32 * x.abs().max()
                    to[i, h] = U_BF16 * o[i, h].abs() + ((U_F16 if ks is not None else U_BF16) + 2 * ds + 2.0 ** -18) * (p @ Vh.abs())
                    tl[i, h] = ds + 2.0 ** -20 * (1 + l[i, h].abs())
        outs.append(o)
        lses.append(l)
        tol_o.append(to)
        tol_l.append(tl)
    return tuple(torch.stack(t) for t in (outs, lses, tol_o, tol_l))


def norm_rope(x, w, rope, pos, eps, inter):
    """[B, N, H, D] in 64 bits, and the largest magnitude met on the way to each element."""
    y = x.double()
    if w is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * w.double()
    mag = y.abs()
    if rope is not None:
        rot = rope.shape[1]
        cs = rope.double()[pos.long()][:, :, None]
        c, s = cs[..., :rot // 2], cs[..., rot // 2:]
        i = torch.arange(rot // 2)
        lo, hi = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
        a, b = y[..., lo].clone(), y[..., hi].clone()
        y[..., lo], y[..., hi] = a * c - b * s, b * c + a * s
        mag[..., lo] = mag[..., hi] = a.abs() + b.abs()
    return y, mag


def rope_table(n, rot):
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    a = torch.arange(n, dtype=torch.float64)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def logprobs(z, tok, K, T):
    """logprob, entropy, top lists of rows [R, V] in 64 bits."""
    x = z.double() / T
    l = torch.log_softmax(x, 1)
    p = l.exp()
    ent = -torch.where(p > 0, p * l, 0.0).sum(1)
    R, V = z.shape
    idx = torch.full((R, K), -1, dtype=torch.int64)
    top = torch.full((R, K), -math.inf, dtype=torch.float64)
    if K:
        order = torch.sort(-(z.double() + 0.0), dim=1, stable=True).indices[:, :K]
        idx[:, :order.shape[1]] = order
        top[:, :order.shape[1]] = l.gather(1, order)
    return l.gather(1, tok.long()[:, None])[:, 0], ent, idx, top

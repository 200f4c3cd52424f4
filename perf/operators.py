"""The target model's side of a verification step, as measurable cases.

Around the verification calls a serving loop runs five more operators on every step: it
normalises and rotates the queries and keys of the drafted positions and writes keys and
values into a paged cache (`kv_append`), attends from those positions over the cache
(`paged_attention`), reports log-probabilities of the emitted tokens (`token_logprobs`),
moves the accepted path of a draft tree to the front of the drafted slots (`kv_compact`),
and reads cached positions back (`kv_read`).

`run` computes each of them in its plain form (elementary torch operations in 32 bits,
rounded once at the end) or, where `own` is true, through this package.
"""
import math

import torch

own = False

FP8_MAX = 448.0          # largest finite e4m3 value
FP8_AMAX_FLOOR = 1e-20   # rows below this quantise with its scale (and so to zero)


def _sv():
    import speculative_decoding_verification_59_gb300 as sv
    return sv


# ---- the cases ------------------------------------------------------------------------
def listed():
    return [
        # One new token of one sequence: the smallest step there is, a single request
        # decoding without drafts.  32 query heads, 8 cached heads of 128.
        dict(name="append-one", op="append", B=1, N=1, Hq=32, Hkv=8, D=128, ctx=777, page=16, fp8=False, rot=128, inter=False, norm=True),
        # 64 sequences of 7 drafts and one more position, cache held in 8 bits; the new
        # positions are read back, as a check or a transfer to another worker does.
        dict(name="append-b64-fp8", op="append", B=64, N=8, Hq=32, Hkv=8, D=128, ctx=200, page=64, fp8=True, rot=128, inter=False, norm=True),
        # One short cached prompt copied out of a bf16 cache with pages of 16.
        dict(name="read-one", op="read", B=1, T=1001, Hkv=8, D=128, page=16, fp8=False),
        # 64 cached contexts of 8 bits handed to another worker as bf16.
        dict(name="read-b64-fp8", op="read", B=64, T=2048, Hkv=8, D=128, page=64, fp8=True),
        # One request decoding one token over a short context: latency.
        dict(name="attend-one", op="attend", B=1, N=1, Hq=32, Hkv=8, D=128, ctx=1000, page=16, fp8=False, tree=False, hnd=False),
        # The ordinary step: 64 sequences of 7 drafts (8 positions), ragged contexts.
        dict(name="attend-chain-b64", op="attend", B=64, N=8, Hq=32, Hkv=8, D=128, ctx=4096, page=64, fp8=False, tree=False, hnd=False),
        # 32 draft trees of 36 nodes (main chain of 7, 4 branches at each depth).
        dict(name="attend-tree-b32", op="attend", B=32, N=36, Hq=32, Hkv=8, D=128, ctx=2048, page=16, fp8=False, tree=True, hnd=False),
        # Few sequences with long contexts in an 8-bit cache, pages laid out head first.
        dict(name="attend-long-fp8", op="attend", B=8, N=8, Hq=32, Hkv=8, D=128, ctx=32768, page=32, fp8=True, tree=False, hnd=True),
        # The accepted path of one 36-node tree moved to the front, 4 layers of a small model.
        dict(name="compact-one", op="compact", B=1, N=36, L=4, Hkv=8, D=64, ctx=30, page=16),
        # The same for 32 trees in all 36 layers of a cache at once.
        dict(name="compact-b32", op="compact", B=32, N=36, L=36, Hkv=8, D=128, ctx=40, page=16),
        # The five positions of one small fp32 chain.
        dict(name="logprobs-small", op="logprobs", rows=5, V=1000, K=2, f32=True, T=1.0),
        # Log-probabilities of all 512 positions of 64 chains, with 5 alternatives each.
        dict(name="logprobs-b64", op="logprobs", rows=512, V=151936, K=5, f32=False, T=0.6),
    ]


def _logint(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "read", "compact", "logprobs", "logprobs"])
    D = rng.choice([64, 128, 128, 256])
    Hkv = rng.choice([1, 2, 4, 8])
    page = rng.choice([8, 16, 32, 48, 64, 128])
    fp8 = rng.random() < 0.5
    if op == "append":
        rot = rng.choice([D, D, D // 2])
        return dict(op=op, B=_logint(rng, 1, 96), N=rng.randint(1, 12), Hq=Hkv * rng.choice([1, 2, 4, 7, 8]), Hkv=Hkv, D=D, ctx=rng.randint(0, 300), page=page,
                    fp8=fp8, rot=rot, inter=rng.random() < 0.3, norm=rng.random() < 0.8)
    if op == "attend":
        tree = rng.random() < 0.35
        N = rng.randint(2, 64) if tree else rng.randint(1, 17)
        G = rng.choice([1, 2, 4, 4, 5, 8])
        B = _logint(rng, 1, 64)
        # at most the cached bytes and the products of the largest listed case
        most = min(2.5e8 / (B * Hkv * D), 1.6e10 / (B * N * Hkv * G * D) / 2, 40000)
        return dict(op=op, B=B, N=N, Hq=Hkv * G, Hkv=Hkv, D=D, ctx=_logint(rng, 1, max(1, int(most))), page=page, fp8=fp8, tree=tree, hnd=rng.random() < 0.5)
    if op == "read":
        B = _logint(rng, 1, 64)
        return dict(op=op, B=B, T=_logint(rng, 1, max(1, int(1.3e8 / (B * Hkv * D)))), Hkv=Hkv, D=D, page=page, fp8=fp8)
    if op == "compact":
        return dict(op=op, B=_logint(rng, 1, 32), N=36, L=rng.randint(1, 36), Hkv=Hkv, D=rng.choice([64, 128]), ctx=rng.randint(0, 60), page=rng.choice([8, 16, 32, 48]))
    f32 = rng.random() < 0.4
    V = _logint(rng, 1000, 151936)
    return dict(op=op, rows=_logint(rng, 1, max(1, int(7.5e7 / V / (2 if f32 else 1)))), V=V, K=rng.randint(0, 8), f32=f32, T=rng.choice([0.6, 1.0, 1.3]))


# ---- inputs ---------------------------------------------------------------------------
def _lens(B, longest):
    """Ragged lengths in [longest/2, longest], the first one the longest."""
    return [longest - (b * 7919) % (longest // 2 + 1) for b in range(B)]


def _tree(N):
    """Parents of a draft tree: a main chain of about N / 5 nodes, the other nodes dealt to
    its nodes as single-node branches.  36 nodes: chain of 7, 4 branches at each depth."""
    depth = max(1, (N - 1) // 5) if N > 1 else 0
    return [-1] + list(range(depth)) + [(n - depth - 1) * depth // max(1, N - 1 - depth) for n in range(depth + 1, N)]


def _depths(parents):
    d = []
    for n, p in enumerate(parents):
        d.append(0 if p < 0 else d[p] + 1)
    return d


def _pool(g, dev, B, tokens, page, Hkv, D, fp8, hnd=False, L=None):
    """A paged cache with random contents: more pages than are in use, dealt out of order."""
    per = -(-tokens // page)
    pages = B * per + 3
    lead = () if L is None else (L,)
    shape = lead + ((pages, Hkv, page, D) if hnd else (pages, page, Hkv, D))
    s = {"page": page, "table": torch.randperm(pages, generator=g, device=dev)[:B * per].view(B, per).to(torch.int32)}
    for name in ("k", "v"):
        if fp8:
            # 8-bit contents with per-row scales, as written by the append: values over the
            # whole e4m3 range, scales that give rows of about unit deviation
            t = torch.empty(shape, device=dev, dtype=torch.float8_e4m3fn)
            flat = t.view(-1, D)
            for lo in range(0, flat.shape[0], 1 << 20):
                flat[lo:lo + (1 << 20)] = (torch.randn(flat[lo:lo + (1 << 20)].shape, generator=g, device=dev) * 110).clamp_(-448, 448).to(torch.float8_e4m3fn)
            sc = (torch.rand(shape[:-1], generator=g, device=dev) + 0.5) / 110
            s[name + "_scale"] = sc.transpose(-1, -2) if hnd else sc
        else:
            t = torch.empty(shape, device=dev, dtype=torch.bfloat16).normal_(generator=g)
            s[name + "_scale"] = None
        s[name] = t.transpose(-2, -3) if hnd else t      # always [..., pages, page, Hkv, D]
    return s


def _cache(s):
    return _sv().KVCache(s["k"], s["v"], s["table"], s["k_scale"], s["v_scale"])


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    c = case
    s = {"op": c["op"], "case": c}
    if c["op"] == "append":
        B, N, D, rot = c["B"], c["N"], c["D"], c["rot"]
        s.update(_pool(g, dev, B, c["ctx"] + N, c["page"], c["Hkv"], D, c["fp8"]))
        s["lens"] = torch.tensor(_lens(B, c["ctx"]), dtype=torch.int32, device=dev)
        # the output of one fused projection: queries, keys and values of a token side by side
        qkv = torch.randn((B, N, c["Hq"] + 2 * c["Hkv"], D), generator=g, device=dev).to(torch.bfloat16)
        s["q"], s["nk"], s["nv"] = qkv.split([c["Hq"], c["Hkv"], c["Hkv"]], dim=2)
        s["qw"] = (torch.rand(D, generator=g, device=dev) + 0.5).to(torch.bfloat16) if c["norm"] else None
        s["kw"] = (torch.rand(D, generator=g, device=dev) + 0.5).to(torch.bfloat16) if c["norm"] else None
        f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
        a = torch.arange(c["ctx"] + N, dtype=torch.float64)[:, None] * f
        s["rope"] = torch.cat([a.cos(), a.sin()], 1).to(torch.float32).to(dev)
    elif c["op"] == "read":
        s.update(_pool(g, dev, c["B"], c["T"], c["page"], c["Hkv"], c["D"], c["fp8"]))
        s["lens"] = torch.tensor(_lens(c["B"], c["T"]), dtype=torch.int32, device=dev)
    elif c["op"] == "attend":
        B, N, D = c["B"], c["N"], c["D"]
        s.update(_pool(g, dev, B, c["ctx"] + N, c["page"], c["Hkv"], D, c["fp8"], c["hnd"]))
        s["lens"] = torch.tensor(_lens(B, c["ctx"]), dtype=torch.int32, device=dev)
        # scores of about two standard deviations, so that the softmax has a shape
        s["q"] = (2 * torch.randn((B, N, c["Hq"], D), generator=g, device=dev)).to(torch.bfloat16)
        s["parents"] = torch.tensor(_tree(N), dtype=torch.int32, device=dev).repeat(B, 1) if c["tree"] else None
    elif c["op"] == "compact":
        B, N = c["B"], c["N"]
        s.update(_pool(g, dev, B, c["ctx"] + N, c["page"], c["Hkv"], c["D"], False, L=c["L"]))
        s["lens"] = torch.tensor(_lens(B, c["ctx"]), dtype=torch.int32, device=dev)
        # accepted paths as the tree verification returns them: part of the main chain, then
        # for most sequences one branch node
        par = _tree(N)
        depth = max(1, (N - 1) // 5)
        path = torch.full((B, N), -1, dtype=torch.int32)
        acc = torch.zeros(B, dtype=torch.int32)
        take = torch.randint(0, depth + 1, (B,), generator=g, device=dev).tolist()
        for b in range(B):
            nodes = list(range(1, take[b] + 1))
            branch = [n for n in range(depth + 1, N) if par[n] == take[b]]
            if branch and b % 4 != 3:
                nodes.append(branch[b % len(branch)])
            path[b, :len(nodes)] = torch.tensor(nodes, dtype=torch.int32)
            acc[b] = len(nodes)
        s["path"], s["acc"] = path.to(dev), acc.to(dev)
    else:
        R, V = c["rows"], c["V"]
        z = torch.randn((R, V), generator=g, device=dev) * 3
        z.scatter_add_(1, torch.randint(0, V, (R, 20), generator=g, device=dev), torch.full((R, 20), 8.0, device=dev))
        # every fourth row belongs to a constrained grammar: a third of its tokens are masked
        z[::4].masked_fill_(torch.rand((len(range(0, R, 4)), V), generator=g, device=dev) < 0.33, -math.inf)
        tok = torch.randint(0, V, (R,), generator=g, device=dev)
        top = z.argmax(1)
        keep = torch.rand(R, generator=g, device=dev) < 0.5      # half the tokens are likely ones
        tok = torch.where(keep | (z.gather(1, tok[:, None])[:, 0] == -math.inf), top, tok)
        s["z"] = z if c["f32"] else z.to(torch.bfloat16)
        s["tok"] = tok.to(torch.int32)
    if own and c["op"] != "logprobs":
        s["cache"] = _cache(s)
    return s


# ---- the plain forms ------------------------------------------------------------------
def _at(s, pos):
    """Pages and slots of positions pos [B, n] of each sequence."""
    p = pos.long()
    return s["table"].long().gather(1, p // s["page"]), p % s["page"]


def _fetch(s, pos, dt):
    """Cached keys and values at positions pos [B, n], as dt: [B, n, Hkv, D] each."""
    pg, sl = _at(s, pos)
    both = []
    for name in ("k", "v"):
        x = s[name][pg, sl].to(dt)
        if s[name + "_scale"] is not None:
            x = x * s[name + "_scale"][pg, sl].to(dt)[..., None]
        both.append(x)
    return both


def _norm_rope(x, w, cs, inter, eps, dt):
    """x [B, N, H, D] normalised over D with weight w, its first rot elements rotated by the
    cosines and sines cs [B, N, rot]."""
    x = x.to(dt)
    if w is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w.to(dt)
    rot = cs.shape[-1]
    co, si = cs[:, :, None, :rot // 2].to(dt), cs[:, :, None, rot // 2:].to(dt)
    head, rest = x[..., :rot], x[..., rot:]
    if inter:
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack([a * co - b * si, b * co + a * si], -1).flatten(-2)
    else:
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        head = torch.cat([a * co - b * si, b * co + a * si], -1)
    return torch.cat([head, rest], -1)


def _plain_append(s):
    c = s["case"]
    pos = s["lens"][:, None] + torch.arange(c["N"], device=s["lens"].device)
    cs = s["rope"][pos.long()]
    q = _norm_rope(s["q"], s["qw"], cs, c["inter"], 1e-6, torch.float32).to(torch.bfloat16)
    k = _norm_rope(s["nk"], s["kw"], cs, c["inter"], 1e-6, torch.float32)
    pg, sl = _at(s, pos)
    if not c["fp8"]:
        s["k"][pg, sl] = k.to(torch.bfloat16)
        s["v"][pg, sl] = s["nv"]
        return {"q": q, "k": s["k"], "v": s["v"]}
    _quantise(s, "k", k, pg, sl)
    _quantise(s, "v", s["nv"].to(torch.float32), pg, sl)
    k, v = _fetch(s, pos, torch.float32)
    return {"q": q, "k_scale": s["k_scale"], "v_scale": s["v_scale"], "k": k.to(torch.bfloat16), "v": v.to(torch.bfloat16)}


def _quantise(s, name, x, pg, sl):
    """One scale for each position and head: the row's largest magnitude over 448."""
    sc = x.abs().amax(-1).clamp_min(FP8_AMAX_FLOOR) / FP8_MAX
    s[name][pg, sl] = (x / sc[..., None]).to(torch.float8_e4m3fn)
    s[name + "_scale"][pg, sl] = sc


def _span(s, T):
    """Positions 0..T-1 of every sequence, and which of them it has."""
    t = torch.arange(T, device=s["lens"].device)[None].expand(len(s["lens"]), T)
    have = t < s["lens"][:, None]
    return torch.where(have, t, 0), have


def _plain_read(s):
    pos, have = _span(s, s["case"]["T"])
    k, v = _fetch(s, pos, torch.float32)
    have = have[..., None, None]
    return {"k": torch.where(have, k, 0.0).to(torch.bfloat16), "v": torch.where(have, v, 0.0).to(torch.bfloat16)}


def _visible(s, T):
    """Which of positions 0..T-1 each new position sees: [B, N, T]."""
    c = s["case"]
    t = torch.arange(T, device=s["lens"].device)[None, None]
    ctx = s["lens"][:, None, None]
    if s["parents"] is None:
        return t <= ctx + torch.arange(c["N"], device=t.device)[None, :, None]
    # ancestors and itself: powers of (identity + one step up)
    step = torch.arange(c["N"], device=t.device)
    up = (s["parents"][:, :, None] == step) | (step[:, None] == step)
    anc = torch.linalg.matrix_power(up.double(), 64) > 0
    d = t - ctx
    m = anc.gather(2, d.clamp(0, c["N"] - 1).expand(-1, c["N"], -1))
    return (d < 0) | (m & (d < c["N"]))


def _plain_attend(s, dt=torch.float32):
    c = s["case"]
    B, N, Hkv, D = c["B"], c["N"], c["Hkv"], c["D"]
    T = c["ctx"] + N
    pos = torch.arange(T, device=s["lens"].device)[None].expand(B, T)
    pos = torch.where(pos < s["lens"][:, None] + N, pos, 0)
    k, v = _fetch(s, pos, dt)
    k, v = k.transpose(1, 2), v.transpose(1, 2)                                   # [B, Hkv, T, D]
    q = s["q"].to(dt).view(B, N, Hkv, -1, D).permute(0, 2, 1, 3, 4)             # [B, Hkv, N, G, D]
    G = q.shape[3]
    sc = (q.reshape(B, Hkv, N * G, D) @ k.transpose(2, 3)).view(B, Hkv, N, G, T) * (1.0 / math.sqrt(D))
    sc = sc.masked_fill(~_visible(s, T)[:, None, :, None, :], -math.inf)
    top = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - top)
    z = p.sum(-1, keepdim=True)
    o = ((p / z).view(B, Hkv, N * G, T) @ v).view(B, Hkv, N, G, D)
    lse = (top + torch.log(z))[..., 0]
    return {"out": o.permute(0, 2, 1, 3, 4).reshape(B, N, Hkv * G, D), "lse": lse.permute(0, 2, 1, 3).reshape(B, N, Hkv * G)}


def _plain_compact(s):
    n = s["path"].shape[1]
    step = torch.arange(1, n + 1, device=s["path"].device)[None]
    live = step <= s["acc"][:, None]
    src = s["lens"][:, None] + torch.where(live, s["path"], 0)
    dst = s["lens"][:, None] + torch.where(live, step, 0)
    (sp, ss), (dp, ds) = _at(s, src), _at(s, dst)
    for name in ("k", "v"):
        s[name][:, dp, ds] = s[name][:, sp, ss]
    return {"k": s["k"], "v": s["v"]}


def _plain_logprobs(s, dt=torch.float32):
    c = s["case"]
    z = s["z"].to(dt)
    x = z / c["T"]
    top = x.amax(1, keepdim=True)
    e = torch.exp(x - top)
    total = e.sum(1, keepdim=True)
    lnz = top + torch.log(total)
    # the entropy sum over p (x - top), masked tokens adding nothing
    w = torch.where(e > 0, e * (x - top), torch.zeros((), dtype=dt, device=z.device)).sum(1, keepdim=True)
    out = {"logprob": (x.gather(1, s["tok"].long()[:, None]) - lnz)[:, 0], "entropy": (torch.log(total) - w / total)[:, 0]}
    if c["K"]:
        # larger logit first, lower index first among equal ones: both in one 64-bit key
        b = (s["z"].to(torch.float32) + 0.0).view(torch.int32).long()
        key = torch.where(b >= 0, b, b ^ 0x7FFFFFFF) * (1 << 32) + (0xFFFFFFFF - torch.arange(c["V"], device=z.device))[None]
        idx = 0xFFFFFFFF - (key.topk(c["K"], dim=1).values & 0xFFFFFFFF)
        out["top_idx"] = idx.to(torch.int32)
        out["top_logprob"] = x.gather(1, idx) - lnz
    return out


def _own(s):
    sv, c = _sv(), s["case"]
    if s["op"] == "append":
        q = sv.kv_append(s["cache"], s["q"], s["nk"], s["nv"], s["lens"], s["rope"], q_weight=s["qw"], k_weight=s["kw"], eps=1e-6, interleaved=c["inter"])
        if not c["fp8"]:
            return {"q": q, "k": s["k"], "v": s["v"]}
        k, v = sv.kv_read(s["cache"], c["N"], starts=s["lens"])
        return {"q": q, "k_scale": s["k_scale"], "v_scale": s["v_scale"], "k": k, "v": v}
    if s["op"] == "read":
        k, v = sv.kv_read(s["cache"], c["T"], counts=s["lens"])
        return {"k": k, "v": v}
    if s["op"] == "attend":
        out, lse = sv.paged_attention(s["q"], s["cache"], s["lens"], parents=s["parents"], lse=True)
        return {"out": out, "lse": lse}
    if s["op"] == "compact":
        sv.kv_compact(s["cache"], s["lens"], s["path"], s["acc"])
        return {"k": s["k"], "v": s["v"]}
    lp, ent, idx, top = sv.token_logprobs(s["z"], s["tok"], c["K"], temperature=c["T"])
    return {"logprob": lp, "entropy": ent, **({"top_idx": idx, "top_logprob": top} if c["K"] else {})}


def run(state):
    if own:
        return _own(state)
    op = state["op"]
    if op == "append":
        return _plain_append(state)
    if op == "read":
        return _plain_read(state)
    if op == "attend":
        r = _plain_attend(state)
        return {"out": r["out"].to(torch.bfloat16), "lse": r["lse"]}
    if op == "compact":
        return _plain_compact(state)
    return _plain_logprobs(state)


# ---- what a pass cannot do without ----------------------------------------------------
def work(case):
    c = case
    if c["op"] == "logprobs":
        e = c["rows"] * c["V"]
        return {"bytes": e * (4 if c["f32"] else 2) + c["rows"] * (12 + 8 * c["K"]), "flops": 6 * e}
    row = c["Hkv"] * (c["D"] + 4 if c.get("fp8") else 2 * c["D"])       # one cached position, keys or values
    if c["op"] == "append":
        tok = c["B"] * c["N"]
        back = 2 * row + 4 * c["Hkv"] * c["D"] if c["fp8"] else 0         # the new positions read back
        return {"bytes": tok * (4 * c["Hq"] * c["D"] + 4 * c["Hkv"] * c["D"] + 2 * row + back + 4 * c["rot"]), "flops": 8 * tok * (c["Hq"] + c["Hkv"]) * c["D"]}
    if c["op"] == "read":
        return {"bytes": sum(_lens(c["B"], c["T"])) * 2 * row + c["B"] * c["T"] * 4 * c["Hkv"] * c["D"], "flops": c["B"] * c["T"] * 2 * c["Hkv"] * c["D"]}
    if c["op"] == "attend":
        n = sum(x + c["N"] for x in _lens(c["B"], c["ctx"]))
        return {"bytes": 2 * n * row + c["B"] * c["N"] * c["Hq"] * (4 * c["D"] + 4), "flops": 4 * n * c["N"] * c["Hq"] * c["D"]}
    # about half a path of each sequence moves; at the least one row of each
    return {"bytes": c["B"] * c["L"] * 4 * row, "flops": 0}


# ---- 64 bits, written apart -----------------------------------------------------------
def _rows(s, name, b, upto):
    """Positions 0..upto-1 of sequence b in 64 bits: [upto, Hkv, D]."""
    page, out = s["page"], []
    pages = s["table"][b, :-(-upto // page)].tolist()
    x = torch.cat([s[name][p] for p in pages])[:upto].to(torch.float64)
    if s[name + "_scale"] is not None:
        x = x * torch.cat([s[name + "_scale"][p] for p in pages])[:upto].to(torch.float64)[..., None]
    return x


def _e4m3(x):
    """The nearest e4m3 value (ties to even), saturating: 3 mantissa bits, least exponent -6."""
    e = torch.floor(torch.log2(x.abs().clamp_min(2.0 ** -30))).clamp(-6, 8)
    step = torch.pow(2.0, e - 3)
    return (torch.round(x / step) * step).clamp(-FP8_MAX, FP8_MAX)


def _exact_rotate(x, w, cs, inter):
    x = x.double()
    if w is not None:
        x = w.double() * x / torch.sqrt(torch.square(x).sum(-1, keepdim=True) / x.shape[-1] + 1e-6)
    rot = cs.shape[-1]
    i = torch.arange(rot // 2, device=x.device)
    lo, hi = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
    z = torch.complex(x[..., lo], x[..., hi]) * torch.complex(cs[..., :rot // 2].double(), cs[..., rot // 2:].double())[:, None]
    y = x.clone()
    y[..., lo], y[..., hi] = z.real, z.imag
    return y


def exact(case, seed):
    s, c = prepare(case, seed), case
    if c["op"] == "compact" or c.get("rows", 0) > 4096:
        return None                               # rows moved as they are; too many rows, one by one
    if c["op"] == "logprobs":
        lp, ent, top = [], [], []
        for r in range(c["rows"]):
            x = s["z"][r].double() / c["T"]
            l = torch.log_softmax(x, 0)
            p = l.exp()
            lp.append(l[int(s["tok"][r])])
            ent.append(-(p * l)[p > 0].sum())
            if c["K"]:
                top.append(l.sort(descending=True).values[:c["K"]])
        return {"logprob": torch.stack(lp), "entropy": torch.stack(ent), **({"top_idx": None, "top_logprob": torch.stack(top)} if c["K"] else {})}
    n, B = s["lens"].tolist(), c["B"]
    if c["op"] == "read":
        both = {}
        for name in ("k", "v"):
            both[name] = torch.zeros((B, c["T"], c["Hkv"], c["D"]), dtype=torch.float64, device=s["table"].device)
            for b in range(B):
                both[name][b, :n[b]] = _rows(s, name, b, n[b])
        return both
    N = c["N"]
    if c["op"] == "append":
        cs = torch.stack([s["rope"][n[b]:n[b] + N] for b in range(B)])
        q, k = (torch.stack([_exact_rotate(s[x][b], s[w], cs[b], c["inter"]) for b in range(B)]) for x, w in (("q", "qw"), ("nk", "kw")))
        new = {"k": k, "v": s["nv"].double()}
        out = {"q": q}
        for name in ("k", "v"):
            sc = new[name].abs().amax(-1).clamp_min(FP8_AMAX_FLOOR) / FP8_MAX
            whole = s[name].double() if not c["fp8"] else None
            scale = s[name + "_scale"].double() if c["fp8"] else None
            for b in range(B):
                for i in range(N):
                    pg, sl = int(s["table"][b, (n[b] + i) // c["page"]]), (n[b] + i) % c["page"]
                    if c["fp8"]:
                        scale[pg, sl] = sc[b, i]
                    else:
                        whole[pg, sl] = new[name][b, i]
            out[name] = _e4m3(new[name] / sc[..., None]) * sc[..., None] if c["fp8"] else whole
            if c["fp8"]:
                out[name + "_scale"] = scale
        return out
    D, Hkv = c["D"], c["Hkv"]
    G = c["Hq"] // Hkv
    par = _tree(N) if c["tree"] else list(range(-1, N - 1))
    outs, lses = [], []
    for b in range(B):
        k, v = _rows(s, "k", b, n[b] + N), _rows(s, "v", b, n[b] + N)
        sees = torch.zeros((N, n[b] + N), dtype=torch.bool)
        for i in range(N):
            sees[i, :n[b]] = True
            a = i
            while a >= 0:
                sees[i, n[b] + a] = True
                a = par[a]
        q = s["q"][b].double().view(N, Hkv, G, D)
        l = torch.einsum("nhgd,thd->hgnt", q, k) / math.sqrt(D)
        l = torch.where(sees.to(l.device), l, -math.inf)
        outs.append(torch.einsum("hgnt,thd->nhgd", torch.softmax(l, -1), v).reshape(N, Hkv * G, D))
        lses.append(torch.logsumexp(l, -1).permute(2, 0, 1).reshape(N, Hkv * G))
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}

"""Greedy decoding with draft trees, from the cache to the tokens' log-probabilities.

A small decoder with random weights (bf16, E4M3 or bf16 cache) generates for B sequences.
Every step runs the calls of this library in the order a serving loop would:

  ngram_retrieve       the main chain of the draft: what followed the last occurrence of the
                       last w tokens
  kv_append            per layer: head norms, rotation by the node's depth, the tree's keys and
                       values into the paged cache behind the verified context
  paged_attention      per layer: each node over the context, its ancestors and itself
  verify_tree_greedy   the longest path of nodes that the decoder agrees with, and one token more
  kv_compact           the path's entries to the front of the tree's slots, all layers at once
  token_logprobs       what the emitted tokens had as probability, the distribution's entropy and
                       its K best tokens, which are the branches when the position is drafted from

The projections are plain matrix products, or, with the weights held in 8 bits, calls of this library
too:

  add_norm             the residual's addition, its norm, rows rounded to 8 bits
  matmul_e4m3          the projections, and the logits
  quantize_e4m3        the attention's output to 8 bits (and, once, the weights)
  gated_act            the activation between the feed-forward products, to 8 bits

Nothing is read back to the host between steps.

  python examples/tree_decode.py [--batch 4] [--steps 24] [--fp8] [--fp8-weights]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_verification_59_gb300 as sv  # noqa: E402


class Decoder:
    """Layers of attention and a gated product, with root-mean-square norms."""
    vocab, dim, heads, kv_heads, head_dim, layers, rows = 512, 256, 8, 2, 64, 2, 4096

    def __init__(self, seed: int = 0, fp8_weights: bool = False):
        g = torch.Generator().manual_seed(seed)

        def w(*shape):
            return (torch.randn(shape, generator=g) * shape[-1] ** -0.5).to(torch.bfloat16).cuda()

        H, G, D = self.heads, self.kv_heads, self.head_dim
        self.embed = (torch.randn((self.vocab, self.dim), generator=g)).to(torch.bfloat16).cuda()
        self.qkv = [w((H + 2 * G) * D, self.dim) for _ in range(self.layers)]
        self.proj = [w(self.dim, H * D) for _ in range(self.layers)]
        self.up = [w(4 * self.dim, self.dim) for _ in range(self.layers)]
        self.down = [w(self.dim, 2 * self.dim) for _ in range(self.layers)]
        self.head = w(self.vocab, self.dim) * 2
        self.q_weight = [torch.ones(D, dtype=torch.bfloat16, device="cuda") for _ in range(self.layers)]
        self.fp8_weights = fp8_weights
        if fp8_weights:
            def quantized(w):
                return sv.quantize_e4m3(w, block_rows=128)
            self.qkv8, self.proj8, self.up8, self.down8 = (
                [quantized(w) for w in ws] for ws in (self.qkv, self.proj, self.up, self.down))
            self.head8 = quantized(self.head)
        angle = torch.arange(self.rows)[:, None] * 10000.0 ** (-torch.arange(D // 2) / (D // 2))
        self.rope = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()

    def cache(self, B: int, tokens: int, page: int = 16, fp8: bool = False) -> sv.KVCache:
        per = -(-tokens // page)
        shape = (self.layers, B * per, page, self.kv_heads, self.head_dim)
        table = torch.randperm(B * per, generator=torch.Generator().manual_seed(1)).view(B, per)
        dtype = torch.float8_e4m3fn if fp8 else torch.bfloat16
        kv = [torch.zeros(shape, dtype=torch.uint8 if fp8 else dtype, device="cuda").view(dtype) for _ in range(2)]
        scale = [torch.ones(shape[:-1], device="cuda") for _ in range(2)] if fp8 else (None, None)
        return sv.KVCache(*kv, table.to(torch.int32).cuda(), *scale)

    @staticmethod
    def norm(x):
        return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)

    def __call__(self, tokens, cache, ctx, parents=None, positions=None):
        """Logits [B, N, vocab] after each of tokens [B, N], which stand at ctx [B] on."""
        if self.fp8_weights:
            return self.forward8(tokens, cache, ctx, parents, positions)
        H, G, D = self.heads, self.kv_heads, self.head_dim
        B, N = tokens.shape
        x = self.embed[tokens.long()]
        for i in range(self.layers):
            part = cache.layer(i)
            q, k, v = (self.norm(x) @ self.qkv[i].T).view(B, N, H + 2 * G, D).split((H, G, G), 2)
            q = sv.kv_append(part, q, k, v, ctx, self.rope, q_weight=self.q_weight[i],
                             k_weight=self.q_weight[i], positions=positions)
            y = sv.paged_attention(q, part, ctx, parents=parents)
            x = x + y.view(B, N, H * D) @ self.proj[i].T
            a, b = (self.norm(x) @ self.up[i].T).chunk(2, -1)
            x = x + (torch.nn.functional.silu(a) * b) @ self.down[i].T
        return (self.norm(x) @ self.head.T).float()

    def forward8(self, tokens, cache, ctx, parents, positions):
        """The same with 8-bit weights: a part's output is added to x by the next norm."""
        H, G, D = self.heads, self.kv_heads, self.head_dim
        B, N = tokens.shape
        x = self.embed[tokens.long()]
        h = sv.add_norm(x, e4m3=True)
        for i in range(self.layers):
            part = cache.layer(i)
            q, k, v = sv.matmul_e4m3(*h, *self.qkv8[i]).view(B, N, H + 2 * G, D).split((H, G, G), 2)
            q = sv.kv_append(part, q, k, v, ctx, self.rope, q_weight=self.q_weight[i],
                             k_weight=self.q_weight[i], positions=positions)
            y = sv.paged_attention(q, part, ctx, parents=parents)
            y = sv.matmul_e4m3(*sv.quantize_e4m3(y.view(B, N, H * D)), *self.proj8[i])
            *h, x = sv.add_norm(y, None, x, e4m3=True)
            y = sv.matmul_e4m3(*sv.gated_act(sv.matmul_e4m3(*h, *self.up8[i]), e4m3=True), *self.down8[i])
            *h, x = sv.add_norm(y, None, x, e4m3=True)
        return sv.matmul_e4m3(*h, *self.head8, dtype=torch.float32)


def generate(model: Decoder, prompt, steps: int, *, chain: int = 6, branches: int = 3, w: int = 2,
             fp8: bool = False):
    """prompt [B, P] int32.  Returns (tokens [B, n], lengths [B], logprobs [B, n], accepted
    [steps, B]): the sequences, their lengths, the emitted tokens' log-probabilities."""
    B, P = prompt.shape
    dev, N = prompt.device, 1 + chain + branches
    room = -(-(P + steps * (chain + 1) + N) // 4) * 4 + 4                    # the last column takes what is dropped
    tokens = torch.zeros((B, room), dtype=torch.int32, device=dev)
    logprobs = torch.zeros((B, room), device=dev)
    best = torch.zeros((B, room, branches), dtype=torch.int32, device=dev)   # of the token after each
    tokens[:, :P] = prompt
    lengths = torch.full((B,), P, dtype=torch.int32, device=dev)
    cache = model.cache(B, room, fp8=fp8)

    # the prompt but for its last token, as chains
    for at in range(0, P - 1, 64):
        part = tokens[:, at:min(at + 64, P - 1)].contiguous()
        logits = model(part, cache, torch.full_like(lengths, at))
        following = tokens[:, at + 1:at + 1 + part.shape[1]].contiguous()
        best[:, at:at + part.shape[1]] = sv.token_logprobs(logits, following, branches)[2]

    # node 0 the last token, then the chain, then other tokens to follow node 0
    parents = torch.tensor([-1] + list(range(chain)) + [0] * branches, dtype=torch.int32, device=dev)
    depth = torch.tensor(list(range(chain + 1)) + [1] * branches, dtype=torch.int32, device=dev)
    parents = parents.repeat(B, 1)
    accepted = []
    row, step = torch.arange(B, device=dev), torch.arange(chain + 1, device=dev)
    for _ in range(steps):
        ctx = lengths - 1
        count, matches, draft = sv.ngram_retrieve(tokens, lengths, w, chain, 64)
        reuse = matches[row, (count.clamp(1, 64) - 1).long()].clamp(min=0).long()
        nodes = torch.cat([tokens[row, ctx.long()][:, None], draft, best[row, reuse]], 1)
        nodes = nodes.clamp(min=0)                                            # no draft: any token
        logits = model(nodes, cache, ctx, parents, ctx[:, None] + depth)
        path, out, acc = sv.verify_tree_greedy(logits, nodes, parents)
        sv.kv_compact(cache, ctx, path, acc)
        # token i came from the logits of node i of the path (node 0 first)
        source = torch.cat([torch.zeros_like(acc)[:, None], path[:, :chain]], 1).clamp(min=0).long()
        rows = logits.gather(1, source[:, :, None].expand(-1, -1, model.vocab))
        out = out[:, :chain + 1].contiguous()
        lp, _, top, _ = sv.token_logprobs(rows, out.clamp(min=0), branches)
        b, i = row[:, None], torch.where(step <= acc[:, None], lengths[:, None] + step, room - 1)
        tokens[b, i], logprobs[b, i], best[b, i - 1] = out, lp, top
        lengths = lengths + acc + 1
        accepted.append(acc)
    error = cache.read_error()
    if error:
        raise RuntimeError(f"cache error bits {error}")
    return tokens, lengths, logprobs, torch.stack(accepted)


def make_prompt(B: int, P: int, vocab: int, seed: int = 0):
    """Random tokens of which a span comes twice."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randint(0, vocab, (B, P), generator=g, dtype=torch.int32)
    x[:, P // 2:P // 2 + P // 4] = x[:, :P // 4]
    return x.cuda()


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--steps", type=int, default=24)
    ap.add_argument("--fp8", action="store_true", help="an 8-bit cache")
    ap.add_argument("--fp8-weights", action="store_true", help="8-bit weights")
    args = ap.parse_args()
    model = Decoder(fp8_weights=args.fp8_weights)
    tokens, lengths, logprobs, accepted = generate(
        model, make_prompt(args.batch, 97, model.vocab), args.steps, fp8=args.fp8)
    for b in range(args.batch):
        n = int(lengths[b])
        print(f"sequence {b}: {n - 97} tokens in {args.steps} steps, mean log-probability "
              f"{logprobs[b, 97:n].mean().item():.3f}, last {tokens[b, n - 8:n].tolist()}")
    print(f"accepted drafts per step: {accepted.float().mean().item():.2f}")


if __name__ == "__main__":
    main()

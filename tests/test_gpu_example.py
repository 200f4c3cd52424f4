"""The decoding example against its decoder in 64 bits, one dense pass over what it emitted."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    import __graft_entry__
    __graft_entry__.build()
    spec = importlib.util.spec_from_file_location("tree_decode", os.path.join(ROOT, "examples", "tree_decode.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def dense(model, tokens):
    """Log-probabilities [n, vocab] after each of tokens [n], in 64 bits from the same weights."""
    H, G, D, n = model.heads, model.kv_heads, model.head_dim, len(tokens)

    def f(t):
        return t.cpu().double()

    def norm(x):
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)
    cos, sin = f(model.rope)[:n, None].chunk(2, -1)

    def turn(x):
        a, b = norm(x).chunk(2, -1)
        return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    x = f(model.embed)[tokens.long()]
    hide = torch.ones(n, n, dtype=torch.bool).triu(1)
    for i in range(model.layers):
        q, k, v = (norm(x) @ f(model.qkv[i]).T).view(n, H + 2 * G, D).split((H, G, G), 1)
        q, k, v = turn(q), turn(k).repeat_interleave(H // G, 1), v.repeat_interleave(H // G, 1)
        p = (torch.einsum("nhd,thd->hnt", q, k) * D ** -0.5).masked_fill(hide, -torch.inf).softmax(-1)
        x = x + torch.einsum("hnt,thd->nhd", p, v).reshape(n, H * D) @ f(model.proj[i]).T
        a, b = (norm(x) @ f(model.up[i]).T).chunk(2, -1)
        x = x + (torch.nn.functional.silu(a) * b) @ f(model.down[i]).T
    return (norm(x) @ f(model.head).T).log_softmax(-1)


# Some 16 roundings to bf16 (2^-9 rms of a value's size 2^-0.5 of the unit) lie on the way to logits
# of standard deviation 2: 2 * 4 * 2^-9 = 0.016 rms, six of them 0.1.  An e4m3 cache adds 2^-5 rms
# of half a step per key and value, averaged over heads and positions: the same again times 4.
@pytest.mark.parametrize("fp8,tol", [(False, 0.1), (True, 0.4)])
def test_tree_decode(ex, fp8, tol):
    model = ex.Decoder(seed=3)
    P, B = 61, 3
    prompt = ex.make_prompt(B, P, model.vocab, seed=4)
    tokens, lengths, logprobs, accepted = ex.generate(model, prompt, 20, fp8=fp8)
    tokens, lengths, logprobs = tokens.cpu(), lengths.cpu(), logprobs.cpu().double()
    assert torch.equal(lengths, P + 20 + accepted.sum(0).cpu().int())
    for b in range(B):
        n = int(lengths[b])
        ref = dense(model, tokens[b, :n - 1])[P - 1:]                         # of tokens P .. n - 1
        got = ref.gather(1, tokens[b, P:n, None].long())[:, 0]
        assert (ref.max(-1).values - got).max() <= 2 * tol, "a token that the decoder would not choose"
        assert (logprobs[b, P:n] - got).abs().max() <= tol

"""The decoding example with 8-bit weights against its decoder in 64 bits with the same weights."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import linear_ref as R  # noqa: E402
from test_gpu_example import dense, ex  # noqa: E402, F401


# A row's rounding to e4m3 is off by 2^-4 / 3^0.5 = 0.036 of its elements' size, rms, and a product passes that
# on as 0.036 of its result's.  Nine products lie on the way to logits of standard deviation 2: rms 2 * 0.036
# * 3 = 0.22, six of them 1.3.  (An 8-bit cache adds less than half of that to two of them.)
@pytest.mark.parametrize("fp8", [False, True])
def test_tree_decode_with_8_bit_weights(ex, fp8):  # noqa: F811
    model = ex.Decoder(seed=3, fp8_weights=True)
    for ws, ws8 in ((model.qkv, model.qkv8), (model.proj, model.proj8), (model.up, model.up8), (model.down, model.down8)):
        for i, w8 in enumerate(ws8):
            ws[i] = R.value(*w8, 128)
    model.head = R.value(*model.head8, 128)
    P, B, tol = 61, 3, 1.3
    prompt = ex.make_prompt(B, P, model.vocab, seed=4)
    tokens, lengths, logprobs, accepted = ex.generate(model, prompt, 12, fp8=fp8)
    tokens, lengths, logprobs = tokens.cpu(), lengths.cpu(), logprobs.cpu().double()
    assert torch.equal(lengths, P + 12 + accepted.sum(0).cpu().int())
    for b in range(B):
        n = int(lengths[b])
        ref = dense(model, tokens[b, :n - 1])[P - 1:]                         # of tokens P .. n - 1
        got = ref.gather(1, tokens[b, P:n, None].long())[:, 0]
        assert (ref.max(-1).values - got).max() <= 2 * tol, "a token that the decoder would not choose"
        assert (logprobs[b, P:n] - got).abs().max() <= tol

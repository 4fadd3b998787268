"""The paged-cache example's tokens against a dense evaluation of each request by itself, in float64 on its dequantised
weights.

The dense form rounds q, K, V and the attention's output to bfloat16 where the example does.  What is left of the
difference is the rounding of the softmax's weights, 2^-8 sum_j w_j |v_j| < 2^-8 for values of unit variance, and outputs
that fall on the other side of a rounding, another 2^-8 |o|: below 2^-7 a value.  They are independent, so a projection with rows of
unit length passes on no more than 2^-7 = 0.008 (rms) per layer; two layers, the MLP's factor of at most 2 between them and the
norms (which divide) leave 0.04 at most of a logit of unit variance, 5 times that for the worst of some 200,000, twice for the
difference of two: a picked token's dense logit is within 0.4 of the largest.  Logits of a context that lacks a page, or the row's own
key, are off by more, which the oracle shows by itself."""
import os
import sys

import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu
WITHIN = 0.4


@pytest.fixture(scope="module")
def example():
    import __graft_entry__

    __graft_entry__.build()
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    import serve_paged_cache

    return serve_paged_cache


class Dense:
    def __init__(self, example, lengths, pages, page_size, seed):
        import oracle

        ex = self.ex = example

        def weight(w):
            return torch.from_numpy(oracle.dequantize(ex.q4.q4_export_blocks(w))).cuda().double()

        # in the order in which serve() draws them
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.embed = torch.randn((ex.VOCAB, ex.HIDDEN), generator=g, device="cuda").double()
        layers = [ex.Layer(g, pages, page_size) for _ in range(ex.LAYERS)]
        head = ex.q4.q4_quantize(torch.randn((ex.VOCAB, ex.HIDDEN), generator=g, device="cuda") * ex.HIDDEN ** -0.5)
        self.prompts = [torch.randint(0, ex.VOCAB, (n,), generator=g, device="cuda") for n in lengths]
        self.layers = [([weight(w) for w in x.qkv], weight(x.o), weight(x.gate), weight(x.up), weight(x.down))
                       for x in layers]
        self.head = weight(head)

    def logits(self, tokens, hidden=None):
        """Logits of a whole sequence, [n, VOCAB]; hidden [n, n]: positions that a row is kept from seeing, as a mistake."""
        ex, n = self.ex, tokens.numel()
        at = torch.arange(n, device="cuda")
        unseen = at > at[:, None]
        if hidden is not None:
            unseen = unseen | hidden

        def r(x):
            return x.to(torch.bfloat16).double()

        x, group = self.embed[tokens], ex.Q_HEADS // ex.KV_HEADS
        for qkv, o, gate, up, down in self.layers:
            q, k, v = (ex.norm(x) @ w.T for w in qkv)
            q, k = r(ex.rotate(q.view(n, -1, ex.D), at)), r(ex.rotate(k.view(n, -1, ex.D), at))
            k, v = (t.view(n, -1, ex.D).repeat_interleave(group, 1) for t in (k, r(v)))
            s = torch.einsum("nhd,mhd->hnm", q, k) * ex.D ** -0.5
            w = torch.softmax(s.masked_fill(unseen, float("-inf")), -1).nan_to_num(0.0)
            x = x + r(torch.einsum("hnm,mhd->nhd", w, v)).reshape(n, -1) @ o.T
            y = ex.norm(x)
            x = x + (torch.nn.functional.silu(y @ gate.T) * (y @ up.T)) @ down.T
        return ex.norm(x) @ self.head.T


@pytest.mark.parametrize("budget,pages,page_size", [(96, 64, 16), (17, 30, 16), (500, 8, 128)])
def test_tokens_are_those_of_a_dense_evaluation(example, budget, pages, page_size):
    lengths, new = [120, 7, 64, 1, 200, 33], 9
    tokens, _, _ = example.serve(lengths, new, pages=pages, page_size=page_size, budget=budget, seed=3)
    dense = Dense(example, lengths, pages, page_size, 3)

    def short(mistake):
        """How far each picked token's logit is below the largest."""
        out = []
        for prompt, picked in zip(dense.prompts, tokens):
            sequence = torch.cat([prompt, picked[:-1]])
            at = torch.arange(sequence.numel(), device="cuda")
            x = dense.logits(sequence, mistake(at) if mistake else None)[prompt.numel() - 1:]
            out.append(x.max(-1).values - x.gather(1, picked[:, None])[:, 0])
        return float(torch.cat(out).max())

    assert short(None) <= WITHIN
    assert short(lambda at: at[:, None] == at) > WITHIN  # a row does not see itself
    assert short(lambda at: (at < 16) & (at[:, None] >= 16)) > WITHIN  # a page is lost

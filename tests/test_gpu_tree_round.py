"""The serving-side operators together: rounds of tree speculative decoding generate what plain greedy decoding does."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
sys.path.insert(0, os.path.join(ROOT, "examples"))

from reject_row_vocab_gb300 import _build  # noqa: E402

_build.build()
import tree_round  # noqa: E402


def _next(m, tokens):
    """Log probabilities behind a token list, in fp64."""
    d = {n: getattr(m, n).double() for n in ("embed", "place", "q", "k", "v", "o", "head")}
    t = torch.tensor(tokens, device="cuda")
    x = d["embed"][t] + d["place"][torch.arange(len(tokens), device="cuda")]
    group = m.heads // m.kv_heads
    q = (x[-1] @ d["q"]).view(m.kv_heads, group, m.dim)
    k, v = (x @ d["k"]).view(-1, m.kv_heads, m.dim), (x @ d["v"]).view(-1, m.kv_heads, m.dim)
    p = torch.softmax(torch.einsum("hgd,thd->hgt", q, k) * m.dim ** -0.5, -1)
    a = torch.einsum("hgt,thd->hgd", p, v).reshape(-1)
    return torch.log_softmax((x[-1] + a @ d["o"]) @ d["head"], 0)


def test_rounds_generate_what_greedy_decoding_does():
    gen = torch.Generator().manual_seed(1)
    prompts = [torch.randint(1000, (n,), generator=gen).tolist() for n in (5, 40, 17, 1)]
    tokens, logprobs, accepted, losses = tree_round.run(prompts, rounds=6)
    m = tree_round.ToyModel()
    for prompt, toks, lps in zip(prompts, tokens, logprobs):
        assert len(toks) >= 6
        for i, (tok, lp) in enumerate(zip(toks, lps)):
            want = _next(m, prompt + toks[:i])
            # the logits are sums of fp32 products of magnitude up to about 1e2, so 1e-3 covers their rounding
            assert want[tok] >= want.max() - 2e-3
            assert abs(float(want[tok]) - lp) < 2e-3
    assert sum(accepted) > 0 and losses[-1] < losses[0]

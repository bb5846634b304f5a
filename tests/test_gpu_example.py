"""The example that runs the serving operators together.  A sequence that went
through the cache step by step, with drafts kept and dropped, has the logits of
the same tokens in one chunk of a new cache.  Both ways round about 10 values a
layer to bf16 (relative 2^-9 rms each at most) at different sums: relative
difference below 4 * sqrt(2 * 10 * layers) * 2^-9; with an e4m3 cache (2^-5 rms
at most, the same codes both ways but where a bf16 neighbour moves one) four
times that.  The decoder's own choice of token is not compared: a draw next to
an edge may fall to either side."""

import math

import pytest
import torch

from examples import speculative_decode as sd
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache,max_draft", [("bf16", 4), ("bf16", 0), ("fp8", 3)])
def test_steps_are_the_chunk(cache, max_draft):
    say(f"speculative decode {cache} {max_draft}")
    c = sd.Config(cache=cache)
    prompts = sd.prompts_of(3, 90, c.vocab, seed=2)
    steps = 6
    make = lambda: sd.Decoder(c, 3, 91 + steps * (max_draft + 1), device=DEV)  # noqa: E731
    d = make()
    logits = d.prefill(prompts)
    assert [len(t) for t in d.tokens] == [len(p) + 1 for p in prompts]
    bound = 4 * math.sqrt(20 * c.layers) * 2.0 ** -9 * (4 if cache == "fp8" else 1)
    for _ in range(steps):
        before = [len(t) for t in d.tokens]
        kept, logits = d.step(max_draft)
        assert all(0 <= n <= max_draft for n in kept)
        assert [len(t) for t in d.tokens] == [b + n + 1 for b, n in zip(before, kept)]
        assert all(0 <= x < c.vocab for t in d.tokens for x in t)
        say(f"  kept {kept}")
    whole = make().prefill([t[:-1] for t in d.tokens])
    err = (whole - logits).norm(dim=1) / whole.norm(dim=1)
    say(f"  relative differences {err.tolist()}, bound {bound:.4f}")
    assert torch.isfinite(logits).all() and (err <= bound).all()


def test_example_refuses_what_does_not_fit():
    c = sd.Config()
    d = sd.Decoder(c, 1, 16, device=DEV)
    with pytest.raises(ValueError):
        d.prefill([[1] * 17])

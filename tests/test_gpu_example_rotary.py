"""The example with rotary positions, a 4-bit cache, penalties and tokens that are
not allowed.

As without positions, a sequence that went through the cache step by step has
the logits of the same tokens in one chunk.  Two more values a layer are rounded
to bf16 (queries and keys after their positions): 4 * sqrt(2 * 12 * layers) *
2^-9, four times that with an e4m3 cache.  In 4 bits a code moves by one where the
bf16 roundings of both ways differ (by 2^-8 of an element) across the middle
between two: with elements a fifth of the range R on average a share of 2^-8 R /
5 / (R / 15) of them, each by R / 15, where the elements' rms is R / 5.5: relative
sqrt(3 * 2^-8) * 5.5 / 15 = 0.04 of keys and of values in each layer, and four
times that as the bound."""

import math

import pytest
import torch

from examples import speculative_decode as sd
from gpu_util import DEV, say

pytestmark = pytest.mark.gpu


def bound_of(c):
    base = 4 * math.sqrt(24 * c.layers) * 2.0 ** -9
    return {"bf16": base, "fp8": 4 * base, "int4": base + 4 * 0.04 * math.sqrt(2 * c.layers)}[c.cache]


@pytest.mark.parametrize("cache,rotary,max_draft", [("bf16", 10000.0, 4), ("fp8", 500.0, 3), ("int4", 10000.0, 3), ("int4", 0.0, 2)])
def test_steps_are_the_chunk(cache, rotary, max_draft):
    say(f"speculative decode {cache} rotary {rotary} {max_draft}")
    c = sd.Config(cache=cache, rotary=rotary, repeats=1.2, presence=0.3, frequency=0.1)
    prompts = sd.prompts_of(3, 90, c.vocab, seed=2)
    make = lambda: sd.Decoder(c, 3, 91 + 6 * (max_draft + 1), device=DEV)  # noqa: E731
    d = make()
    d.prefill(prompts)
    for _ in range(6):
        kept, logits = d.step(max_draft)
        say(f"  kept {kept}")
    whole = make().prefill([t[:-1] for t in d.tokens])
    err = (whole - logits).norm(dim=1) / whole.norm(dim=1)
    say(f"  relative differences {err.tolist()}, bound {bound_of(c):.4f}")
    assert torch.isfinite(logits).all() and (err <= bound_of(c)).all()


def test_positions_tell_orders_apart():
    """Without positions a last token sees a set; with them a sequence."""
    say("positions")
    for rotary in (0.0, 10000.0):
        c = sd.Config(layers=1, rotary=rotary)  # one layer: what the others see does not reach the last
        a = sd.Decoder(c, 1, 64, device=DEV).prefill([[5, 6, 7, 8, 9, 3]])
        b = sd.Decoder(c, 1, 64, device=DEV).prefill([[9, 7, 8, 5, 6, 3]])
        err = float((a - b).norm() / a.norm())
        say(f"  base {rotary}: {err:.4f}")
        if rotary:
            assert err > 0.02
        else:
            assert err <= 4 * math.sqrt(20) * 2.0 ** -9   # the same values, summed in another order


def test_penalties_and_banned_tokens():
    """Tokens that are not allowed are never drawn, and a large penalty for
    presence leaves no token twice."""
    say("penalties")
    banned = tuple(range(0, 1031, 2))
    c = sd.Config(presence=1e4, banned=banned, cache="int4", rotary=10000.0)
    prompts = sd.prompts_of(4, 40, c.vocab, seed=5)
    d = sd.Decoder(c, 4, 200, device=DEV)
    d.prefill(prompts)
    for _ in range(12):
        d.step(3)
    for t, p in zip(d.tokens, prompts):
        made = t[len(p):]
        assert len(made) == len(set(made)) >= 13 and all(x % 2 for x in made)

"""GPU parity of the token probabilities.

Bounds, e = 2^-24: an adjusted logit is three or four roundings of numbers that
are at most `size` (the sum of the magnitudes that go into it; a quotient or
product by `repeats` keeps relative errors): off by at most 5 e size.  The
exponent (x - top) / temperature has that of both, and 4 e of itself (the
difference, the factor's quotient and product, exp2's argument); the exponential
and the quotient 4 e more, and a sum of n terms, of which each passes at most 24
+ n / 4096 additions of 16 or more at a time, 64 e.  Twice the exponent's error
(weight and sum), all relative to p; below the smallest normal number nothing is
said.  bf16: half a step, 2^-8, more.
"""

import math

import numpy as np
import pytest
import torch

import oracle
from gpu_util import DEV, host_f64, say
from ternary_weights_hadamard_amd import tb

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
S = oracle.serving


def ints(v):
    return torch.tensor(np.asarray(v, dtype=np.int64).astype(np.int32), device=DEV)


class Case:
    def __init__(self, n, vocab, kind=torch.float32, history=30, bias=5, masks=True, seed=0, spread=3.0):
        rng = np.random.default_rng(seed + vocab + len(n))
        self.n, self.vocab, self.b = n, vocab, len(n)
        self.cu = np.concatenate([[0], np.cumsum(n)])
        self.total = int(self.cu[-1])
        self.rows, self.max_draft = self.total + self.b, max(n)
        self.logits = torch.from_numpy(rng.normal(size=(self.rows, vocab)) * spread).to(kind).to(DEV)
        few = max(vocab // 7, 1)                            # tokens come again
        self.drafts = rng.integers(0, few, self.total)
        self.history = [rng.integers(0, few, rng.integers(0, history + 1)).tolist() for _ in n]
        self.prompt = [int(rng.integers(0, len(h) + 1)) for h in self.history]
        self.bias = [[(int(i), float(np.float32(v))) for i, v in zip(rng.integers(0, vocab, bias), rng.normal(size=bias) * 4)]
                     for _ in n]
        self.params = np.stack([rng.uniform(0.3, 1.5, self.b), rng.uniform(0.7, 1.6, self.b), rng.uniform(-1, 1, self.b),
                                rng.uniform(-0.5, 0.8, self.b)], 1).astype(np.float32)
        self.params[1::3, 0] = 0.0                          # the largest is taken
        self.masks = self.mask_row = None
        if masks:
            self.masks = rng.random((3, vocab)) < np.array([0.5, 0.03, 0.0])[:, None]
            self.masks[1, vocab // 2] = True
            self.mask_row = rng.integers(-1, 3, self.rows)

    def mask_words(self):
        words = -(-self.vocab // 32)
        bits = np.zeros((len(self.masks), words * 32), np.uint8)
        bits[:, :self.vocab] = self.masks
        return torch.from_numpy(np.packbits(bits, axis=1, bitorder="little").view(np.int32).copy()).to(DEV)

    def lists(self):
        cat = lambda x: [i for y in x for i in y]  # noqa: E731
        off = lambda x: ints(np.concatenate([[0], np.cumsum([len(y) for y in x])]))  # noqa: E731
        kw = dict(history=ints(cat(self.history)), cu_history=off(self.history), prompt_len=ints(self.prompt),
                  bias=(ints([i for i, _ in cat(self.bias)]),
                        torch.tensor([v for _, v in cat(self.bias)], dtype=torch.float32, device=DEV), off(self.bias)))
        if self.masks is not None:
            kw.update(mask=self.mask_words(), mask_row=ints(self.mask_row))
        return kw

    def run(self, **kw):
        a = dict(drafts=ints(self.drafts), cu_draft=ints(self.cu), max_draft=self.max_draft, **self.lists())
        a.update(kw)
        return tb.tb_token_probs(self.logits, torch.from_numpy(self.params).to(DEV), **a)

    def allowed(self):
        if self.masks is None:
            return [None] * self.rows
        return [self.masks[m] if 0 <= m < 3 else None for m in self.mask_row]

    def reference(self):
        return S.token_probs(host_f64(self.logits), self.params, self.drafts, self.cu, self.max_draft, self.history, None,
                             self.prompt, self.bias, self.allowed())

    def check(self, p, what=""):
        torch.cuda.synchronize()
        got, ref = host_f64(p), self.reference()
        logits, worst = host_f64(self.logits), 0.0
        for b in range(self.b):
            t, repeats, presence, frequency = (float(x) for x in self.params[b])
            most = max([abs(v) for _, v in self.bias[b]] + [0.0])
            times = len(self.history[b]) + self.max_draft
            for row in range(self.cu[b] + b, self.cu[b + 1] + b + 1):
                if t <= 0:
                    assert np.array_equal(got[row], ref[row]), f"{what}: row {row}"
                    continue
                size = (np.abs(logits[row]).max() + most) * max(1.0, repeats, 1 / repeats) + abs(presence) + abs(frequency) * times
                with np.errstate(divide="ignore"):
                    gap = -np.log(np.where(ref[row] > 0, ref[row], 1.0))   # at least (top - x) / t, up to the sum
                bound = (2 * (10 * E * size / t + 4 * E * (gap + math.log(self.vocab))) + 72 * E) * ref[row] + 2.0 ** -120
                if p.dtype == torch.bfloat16:
                    bound = bound + 2.0 ** -8 * ref[row]
                err = np.abs(got[row] - ref[row])
                worst = max(worst, float(np.max(err / bound)))
                assert np.all(err <= bound), f"{what}: row {row}"
        say(f"  {what}: worst error {worst:.2f} of its bound")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,vocab", [([0], 1), ([0, 2], 3), ([3], 31), ([0, 4, 1], 1000), ([2, 0], 4096), ([1], 4097),
                                     ([0, 8], 8195), ([3, 1], 16390), ([2, 5, 0], 32768), ([1, 3], 32769), ([8, 0, 5], 50001),
                                     ([2], 131073)])
def test_matches_oracle(n, vocab, kind, dtype):
    say(f"probs {n} {vocab} {kind} {dtype}")
    c = Case(n, vocab, kind)
    c.check(c.run(out_dtype=dtype), "all")


@pytest.mark.parametrize("vocab", [777, 40001])
def test_parts_alone(vocab):
    """Without drafts, history, bias or masks, and with each alone."""
    say(f"probs parts {vocab}")
    c = Case([0, 0, 0, 0], vocab)
    all_of, lists = (c.history, c.prompt, c.bias, c.masks, c.mask_row), c.lists()
    for keep in ("", "history", "bias", "mask"):
        c.history, c.prompt, c.bias, c.masks, c.mask_row = [[]] * 4, [0] * 4, [[]] * 4, None, None
        kw = dict(drafts=None, cu_draft=None, history=None, cu_history=None, prompt_len=None, bias=None, mask=None, mask_row=None)
        if keep == "history":
            c.history, c.prompt = all_of[0], all_of[1]
            kw.update({k: lists[k] for k in ("history", "cu_history", "prompt_len")})
        if keep == "bias":
            c.bias = all_of[2]
            kw["bias"] = lists["bias"]
        if keep == "mask":
            c.masks, c.mask_row = all_of[3], all_of[4]
            kw.update(mask=lists["mask"], mask_row=lists["mask_row"])
        p = tb.tb_token_probs(c.logits, torch.from_numpy(c.params).to(DEV), **kw)
        c.check(p, keep or "nothing")
    c.history, c.prompt, c.bias, c.masks, c.mask_row = all_of
    c.prompt = [0] * 4                                      # no lengths: all of it was generated
    c.check(c.run(prompt_len=None), "no prompt")
    c.masks, c.mask_row = np.random.default_rng(0).random((4, vocab)) < 0.3, np.arange(4)
    c.allowed = lambda: list(c.masks)
    c.check(c.run(mask_row=None, mask=c.mask_words()), "a mask for each row")


@pytest.mark.parametrize("vocab", [900, 33000])
def test_strides(vocab):
    """Rows inside larger ones, at odd elements; what lies between stays."""
    say(f"probs strides {vocab}")
    c = Case([2, 0, 3], vocab, torch.bfloat16)
    wide = torch.full((c.rows, vocab + 13), 50.0, dtype=torch.bfloat16, device=DEV)
    wide[:, 5:5 + vocab] = c.logits
    c.logits = wide[:, 5:5 + vocab]
    p = torch.full((c.rows, vocab + 7), 3.0, device=DEV)
    words = torch.zeros((3, -(-vocab // 32) + 5), dtype=torch.int32, device=DEV)
    words[:, 3:3 + -(-vocab // 32)] = c.mask_words()
    out = c.run(p=p[:, 3:3 + vocab], mask=words[:, 3:])
    c.logits = c.logits.contiguous()
    c.check(out, "strided")
    assert (p[:, :3] == 3.0).all() and (p[:, 3 + vocab:] == 3.0).all()


@pytest.mark.parametrize("vocab", [900, 33000])
def test_special_logits(vocab):
    say(f"probs special {vocab}")
    inf, nan = float("inf"), float("nan")
    logits = torch.randn(8, vocab, device=DEV)
    masks = np.ones((1, vocab), bool)
    masks[0, [3, vocab - 1]] = False
    c = Case([0], vocab)
    c.masks = masks
    mask = c.mask_words()
    logits[0, 3], logits[0, vocab - 1] = nan, inf          # not allowed: they do not reach the row
    logits[1, :] = -inf                                    # nothing is left
    logits[2, 5] = -inf
    logits[3, 7] = nan                                     # as in the formula
    logits[4, 7] = inf
    logits[5] = -torch.finfo(torch.float32).max            # all equal, the lowest there is
    logits[6, 2] = torch.finfo(torch.float32).max
    logits[7, 100:103], logits[7, 99] = 100.0, nan
    rows = ints([0] + [-1] * 7)
    params = torch.tensor([[0.7, 1.0, 0.0, 0.0]] * 8, device=DEV)
    p = tb.tb_token_probs(logits, params, mask=mask, mask_row=rows)
    ok = torch.isfinite(p).all(dim=1)
    assert ok.tolist() == [True, True, True, False, False, True, True, False]
    sums = p.double().sum(1)
    assert (p[1] == 0).all() and torch.allclose(sums[[0, 2, 5, 6]], torch.ones(4, dtype=torch.float64, device=DEV), atol=1e-5)
    assert p[0, 3] == 0 and p[0, vocab - 1] == 0 and p[2, 5] == 0 and p[6, 2] == 1.0
    assert torch.allclose(p[5], torch.full((vocab,), 1.0 / vocab, device=DEV), rtol=1e-5, atol=0)
    params[:, 0] = 0.0
    p = tb.tb_token_probs(logits, params, mask=mask, mask_row=rows)
    want = torch.zeros_like(p)
    clean = torch.where(torch.isnan(logits), -inf, logits)
    clean[0, 3] = clean[0, vocab - 1] = -inf
    hot = clean.argmax(1)
    hot[5], hot[7] = 0, 100                                # ties: the first
    want[torch.arange(8), hot] = 1.0
    want[1] = 0.0
    assert torch.equal(p, want)
    # a temperature that is no number takes the largest; one without end makes all equal
    params[:, 0] = nan
    assert torch.equal(tb.tb_token_probs(logits, params, mask=mask, mask_row=rows), want)
    params[:, 0] = inf
    p = tb.tb_token_probs(logits[5:7], params[5:7])
    assert torch.allclose(p, torch.full_like(p, 1.0 / vocab), rtol=1e-5, atol=0)
    params[:, 0] = 1e-40                                   # all but the largest vanish
    p = tb.tb_token_probs(logits[6:7], params[6:7])
    assert p[0, 2] == 1.0 and p.sum() == 1.0


@pytest.mark.parametrize("vocab", [900, 33000])
def test_lists_with_wrong_entries(vocab):
    """Ids outside the vocabulary are passed over, offsets are clamped, masks that do not exist allow all."""
    say(f"probs wrong entries {vocab}")
    c = Case([2, 1], vocab, masks=True)
    good = c.run()
    a = c.lists()
    kw = dict(drafts=ints(c.drafts), cu_draft=ints(c.cu), max_draft=c.max_draft)
    # the same lists with ids in between that are none
    wide = lambda t: torch.stack([t, torch.full_like(t, -3)], 1).flatten()  # noqa: E731
    b2 = dict(a)
    b2["history"], b2["cu_history"], b2["prompt_len"] = wide(a["history"]), 2 * a["cu_history"], 2 * a["prompt_len"]
    ids, values, cu = a["bias"]
    b2["bias"] = (torch.where(wide(ids) < 0, vocab + 5, wide(ids)), torch.stack([values, values + 9], 1).flatten(), 2 * cu)
    params = torch.from_numpy(c.params).to(DEV)
    assert torch.equal(tb.tb_token_probs(c.logits, params, **kw, **b2), good)
    # offsets that lead outside, or fall
    far = dict(a, cu_history=ints([-5, 10 ** 9, 3]), prompt_len=ints([10 ** 9, -4]))
    p = tb.tb_token_probs(c.logits, params, **kw, **far)
    c.history, c.prompt = [[i for h in c.history for i in h], []], [10 ** 9, 0]
    c.check(p, "clamped history")
    out = torch.full_like(good, 5.0)
    tb.tb_token_probs(c.logits, params, ints(c.drafts), ints([1, 10 ** 6, -1]), 2, p=out, **a)
    assert torch.isfinite(out).all() and (out[0] == 5.0).all()   # row 0 is no sequence's
    c.mask_row = np.full(c.rows, 77)
    c.check(c.run(**dict(far, mask_row=ints(c.mask_row))), "no such mask")


def test_more_drafts_than_are_looked_at():
    say("probs max_draft")
    c = Case([5, 2], 500)
    c.max_draft = 3
    p = torch.full((c.rows, 500), 5.0, device=DEV)
    c.run(p=p)
    assert (p[4:6] == 5.0).all() and (p[:4] != 5.0).all() and (p[6:] != 5.0).all()


def test_counts_do_not_depend_on_order():
    """The last bias of an id counts, counts are whole numbers: equal calls give equal bits."""
    say("probs order")
    for vocab in (700, 35000):
        c = Case([4, 4, 4], vocab, history=4000, bias=2047, seed=9)
        a = c.run()
        c.check(a, "many")
        for _ in range(3):
            assert torch.equal(c.run(), a)
    # more biases than are looked at: the first 2047
    c = Case([0], 5000, history=0, masks=False, bias=3000, seed=1)
    p = c.run()
    c.bias = [c.bias[0][:2047]]
    c.check(p, "2047 of 3000")


def test_long_history():
    """A count past 2^20: the last generated tokens are counted, the prompt's all noted."""
    say("probs long history")
    n = (1 << 20) + 500
    c = Case([1], 64, history=0, bias=0, masks=False)
    c.params[:] = [1.0, 1.3, 0.1, 1e-6]
    early, most = 7, (1 << 20) - 65
    history = torch.full((n + 1,), 3, dtype=torch.int32, device=DEV)
    history[0] = early                                      # the prompt
    history[1:101] = 9                                      # generated, but too long ago
    p = tb.tb_token_probs(c.logits, torch.from_numpy(c.params).to(DEV), ints([9]), ints([0, 1]), 1, history=history,
                          cu_history=ints([0, n + 1]), prompt_len=ints([1]))
    c.drafts, c.history, c.prompt = np.array([9]), [[early] + [3] * most], [1]
    c.check(p, "long")
    # the most that a count can come to: all of them and 64 drafts the same
    c = Case([64], 64, history=0, bias=0, masks=False)
    c.bias = [[(3, 2.5), (9, 1.5)]]
    c.params[:] = [1.0, 1.3, 0.1, 1e-6]
    c.drafts, c.history, c.prompt = np.full(64, 3), [[early] + [3] * most], [1]
    c.check(c.run(history=history, cu_history=ints([0, n + 1]), prompt_len=ints([1])), "largest count")


def test_feeds_the_verification():
    """Probabilities and the verification of drafts, as they run together: greedy
    sequences keep a draft exactly if it is the largest."""
    say("probs and verify")
    for vocab in (1031, 40000):
        c = Case([3, 3, 0], vocab, masks=False, history=10)
        c.params[:, 0] = 0.0
        ref = c.reference()
        c.drafts[:2] = [int(np.argmax(ref[0])), 1]
        ref = c.reference()
        c.drafts[1] = int(np.argmax(ref[1]))
        ref = c.reference()
        p = c.run()
        u = torch.full((6,), 0.5, device=DEV)
        accepted, tokens = tb.tb_verify_draft(p, None, ints(c.drafts), u, torch.full((3,), 0.5, device=DEV), ints(c.cu), 3)
        lo = 0
        for b in range(3):
            want = []
            for j in range(c.n[b] + 1):
                want.append(int(np.argmax(ref[c.cu[b] + b + j])))
                if j < c.n[b] and c.drafts[c.cu[b] + j] != want[-1]:
                    break
            assert accepted[b] == len(want) - 1 and tokens[b, :len(want)].tolist() == want
        # a row that nothing is allowed in draws nothing
        none = torch.zeros((1, -(-vocab // 32)), dtype=torch.int32, device=DEV)
        p = tb.tb_token_probs(c.logits[:1], torch.from_numpy(c.params[:1]).to(DEV), mask=none)
        accepted, tokens = tb.tb_verify_draft(p, None, ints([]), u[:0], u[:1], ints([0, 0]), 0)
        assert accepted.item() == 0 and tokens.item() == -1


@pytest.mark.parametrize("vocab", [2000, 40000])
def test_streams_and_graphs(vocab):
    say(f"probs streams and graphs {vocab}")
    c = Case([2, 4], vocab)
    want = c.run()
    a = dict(drafts=ints(c.drafts), cu_draft=ints(c.cu), max_draft=c.max_draft, **c.lists())
    params = torch.from_numpy(c.params).to(DEV)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    p = tb.tb_token_probs(c.logits, params, stream=side, **a)
    side.synchronize()
    assert torch.equal(p, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        p = tb.tb_token_probs(c.logits, params, **a)
    keep = c.logits.clone()
    for k in range(3):
        c.logits.copy_(keep * (1 + k))
        eager = c.run()
        p.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(p, eager)


def test_refusals():
    c = Case([1], 100)
    params = torch.from_numpy(c.params).to(DEV)
    i = ints([0, 1])
    with pytest.raises(ValueError):
        tb.tb_token_probs(c.logits, params)                 # a row too many without drafts
    with pytest.raises(ValueError):
        tb.tb_token_probs(c.logits, params, ints([1]), None, 1)
    with pytest.raises(ValueError):
        tb.tb_token_probs(c.logits, params.double(), ints([1]), i, 1)
    with pytest.raises(ValueError):
        tb.tb_token_probs(c.logits, params, ints([1]), i, 1, history=ints([3]))
    with pytest.raises(ValueError):
        tb.tb_token_probs(c.logits, params, ints([1]), i, 1, mask=ints([[1, 2, 3]]))
    with pytest.raises(ValueError):
        tb.tb_token_probs(c.logits, params, ints([1]), i, 1, mask_row=ints([0, 0]))
    with pytest.raises(tb.TBError):
        tb.tb_token_probs(c.logits, params, ints([1]), i, 65)
    with pytest.raises(tb.TBError):
        tb.tb_token_probs(c.logits, params, ints([1]), i, 1, p=c.logits)
    with pytest.raises(TypeError):
        tb.tb_token_probs(c.logits.double(), params, ints([1]), i, 1)

"""Attention over the paged cache where batches, scores and values are not the
usual ones, against the oracle and with the bounds of test_gpu_paged.py."""

import numpy as np
import pytest
import torch

from gpu_util import DEV, say
from test_gpu_paged import Case
from ternary_weights_hadamard_amd import tb

pytestmark = pytest.mark.gpu


def _attend_into(c, q, workspace, **kw):
    """out and lse of q's rows, NaN and 9 where nothing was written."""
    out = torch.full((q.shape[0], c.hq, c.d), float("nan"), device=DEV)
    lse = torch.full((q.shape[0], c.hq), 9.0, device=DEV)
    if not workspace:
        kw["workspace"] = torch.empty(16, dtype=torch.uint8, device=DEV)
    tb.tb_paged_attention(q, c.k, c.v, c.table_d, c.cu_d, c.kv_d, c.max_q, c.max_kv, k_scale=c.k_scale, v_scale=c.v_scale,
                          out=out, lse=lse, **kw)
    torch.cuda.synchronize()
    return out, lse


# ---------------------------------------------------- lengths that the host does not know

@pytest.mark.parametrize("cache", ["bf16", "fp8"])
@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("lens,hq,hkv,extra", [
    ([(32, 50), (8, 40)], 2, 2, 24),                      # as many rows as 2 x 32 tokens, 24 of them of no sequence
    ([(32, 50), (8, 40)], 2, 2, 100),                     # more
    ([(150, 900), (1, 700), (3, 1200)], 5, 1, 297),       # positions in parts
    ([(150, 900), (1, 700), (0, 30), (3, 1200)], 5, 1, 1000),
    ([(9, 300), (2, 2), (9, 40)], 4, 2, 7),
])
def test_rows_of_no_sequence_hide_none(lens, hq, hkv, extra, workspace, cache):
    """The token arrays may have more rows than the sequences have tokens: how many says nothing of the lengths."""
    say(f"padded {lens} {hq} {hkv} {extra} {workspace} {cache}")
    c = Case(lens, hq, hkv, 64, 16, cache)
    q = torch.cat([c.q, torch.full((extra, hq, 64), float("nan"), dtype=torch.bfloat16, device=DEV)])
    out, lse = _attend_into(c, q, workspace)
    c.check(out[:c.total], lse[:c.total], what="padded")
    assert torch.isnan(out[c.total:]).all() and (lse[c.total:] == 9.0).all()


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
@pytest.mark.parametrize("workspace", [True, False])
def test_sequences_past_max_q_hide_none(workspace, cache):
    """A sequence of more than max_q tokens has its first max_q computed; one of few is there beside it."""
    say(f"past max_q {workspace} {cache}")
    c = Case([(60, 400), (4, 300), (30, 33)], 2, 2, 64, 16, cache)
    c.max_q = 17
    out, lse = _attend_into(c, c.q, workspace)
    done = torch.zeros(c.total, dtype=torch.bool, device=DEV)
    for first, n in ((0, 17), (60, 4), (64, 17)):
        done[first:first + n] = True
    assert torch.isnan(out[~done]).all() and (lse[~done] == 9.0).all()
    ref, rl, _, _ = c.reference()
    out[~done] = torch.from_numpy(ref).to(torch.float32).to(DEV)[~done]
    lse[~done] = torch.from_numpy(rl).to(torch.float32).to(DEV)[~done]
    c.check(out, lse, what="past max_q")


# ---------------------------------------------------------------- a dominant score

@pytest.mark.parametrize("cache", ["bf16", "fp8"])
@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("n", [1, 5, 40])
@pytest.mark.parametrize("gap", [12.0, 16.0])
def test_small_weights_beside_a_dominant_one(gap, n, workspace, cache):
    """One position scores `gap` above every other, and its value is 0: the output
    is what the others' small weights make it.  The bound is relative to that."""
    say(f"dominant {gap} {n} {workspace} {cache}")
    kv = 8192
    for at in (0, 5003):
        c = Case([(n, kv)], 2, 1, 128, 64, cache, poison=False)
        g = torch.Generator().manual_seed(n)
        score = torch.randn(kv, generator=g)
        score[at] = score.max() + gap
        k_scale = 1.0 if c.k_scale is None else float(c.k_scale[0])
        # scores are 8 times channel 0 of the keys
        c.q.zero_()
        c.q[:, :, 0] = 8.0
        for x in range(0, kv, c.page):
            i = int(c.table[0, x // c.page])
            c.k[i, 0, :, 0] = (score[x:x + c.page] / 8 / k_scale).to(c.k.dtype).to(DEV)
        c.v[int(c.table[0, at // c.page]), 0, :, at % c.page] = 0.0
        out, lse = _attend_into(c, c.q, workspace, scale=1.0)
        c.check(out, lse, scale=1.0, what=f"{gap} above, at {at}")


# ---------------------------------------------------------------- many sequences

@pytest.mark.parametrize("cache", ["bf16", "fp8"])
@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("kind", ["mixed", "chunks", "steps"])
def test_more_sequences_than_lanes(kind, workspace, cache):
    """More than 64 and more than 256 sequences, some without tokens, of one kind and of both."""
    say(f"many sequences {kind} {workspace} {cache}")
    rng = np.random.default_rng(3)
    lens = []
    for i in range(300 if kind == "chunks" else 130):
        n = {"steps": 1, "chunks": int(rng.integers(9, 14)), "mixed": 1 if i % 9 else int(rng.integers(9, 150))}[kind]
        n = 0 if i % 17 == 4 else n
        lens.append((n, n + int(rng.integers(0, 40 if kind == "chunks" else 900))))
    c = Case(lens, 4, 2, 64, 16, cache)
    out, lse = _attend_into(c, c.q, workspace)
    c.check(out, lse, what=kind)


def _shared_pages(kv, hkv, page):
    """Caches of as many pages as the longest sequence has: all sequences share them."""
    pages, g = -(-kv // page), torch.Generator(device=DEV).manual_seed(5)
    k = torch.randn((pages, hkv, page, 64), generator=g, device=DEV, dtype=torch.bfloat16)
    v = torch.randn((pages, hkv, 64, page), generator=g, device=DEV, dtype=torch.bfloat16)
    return k, v, torch.arange(pages, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("b,long,max_q,window", [(8192, 200, 1 << 20, 0), (256, 131072, 131072, 16), (2, 300, 1 << 21, 0)])
def test_one_prompt_among_many_steps(b, long, max_q, window):
    """As many workgroups as there is work for, however large B and max_q are:
    the prompt (first or last) and the single tokens are what they are alone."""
    hq, hkv, page = 64, 8, 64
    say(f"one prompt of {long} among {b - 1}, max_q {max_q}")
    k, v, pages = _shared_pages(long, hkv, page)
    table = pages.expand(b, -1).contiguous()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    g = torch.Generator(device=DEV).manual_seed(b)
    q = torch.randn((long + b - 1, hq, 64), generator=g, device=DEV, dtype=torch.bfloat16)
    steps = [1 + (7 * i) % 200 for i in range(b - 1)]
    prompt, pl = tb.tb_paged_attention(q[:long], k, v, table[:1], i32([0, long]), i32([long]), long, 250, window=window,
                                       with_lse=True)
    single, sl = tb.tb_paged_attention(q[long:], k, v, table[1:], i32(list(range(b))), i32(steps), 1, 250, window=window,
                                       with_lse=True)
    out, lse = tb.tb_paged_attention(q, k, v, table, i32([0] + list(range(long, long + b))), i32([long] + steps), max_q, 250,
                                     window=window, with_lse=True)
    torch.cuda.synchronize()
    assert torch.equal(out[:long], prompt) and torch.equal(lse[:long], pl)
    assert torch.equal(out[long:], single) and torch.equal(lse[long:], sl)
    turned = torch.cat([q[long:], q[:long]])
    out, lse = tb.tb_paged_attention(turned, k, v, table, i32(list(range(b)) + [long + b - 1]), i32(steps + [long]), max_q, 250,
                                     window=window, with_lse=True)
    torch.cuda.synchronize()
    assert torch.equal(out[b - 1:], prompt) and torch.equal(lse[b - 1:], pl)
    assert torch.equal(out[:b - 1], single) and torch.equal(lse[:b - 1], sl)


# ---------------------------------------------------------- infinities that are seen

@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("scale", [None, 3.0])
@pytest.mark.parametrize("n,kv", [(1, 1000), (12, 1000), (150, 1000)])
def test_infinite_values_stay_infinite(n, kv, scale, workspace):
    """An infinity among the values of a position that a row sees is one in its
    output, however small its weight (scores of scale 3 are hundreds apart); two of
    different signs are NaN.  Other channels and heads are as they were."""
    say(f"infinite {n} {kv} {scale} {workspace}")
    c = Case([(n, kv), (n, n)], 4, 2, 128, 16, "bf16")
    kw = {} if scale is None else dict(scale=scale)
    first, fl = _attend_into(c, c.q, workspace, **kw)
    for places in ([(3, 7, 1)], [(3, 7, -1), (700, 9, 1)], [(0, 7, 1), (517, 7, -1), (400, 9, 1), (401, 9, 1)]):
        d = Case([(n, kv), (n, n)], 4, 2, 128, 16, "bf16")
        want = {}
        for x, ch, sign in places:
            d.v[int(d.table[0, x // 16]), 1, ch, x % 16] = sign * float("inf")
            want[ch] = want.get(ch, 0.0) + sign * float("inf")
        out, lse = _attend_into(d, d.q, workspace, **kw)
        assert torch.equal(lse, fl)
        assert torch.equal(out[n:], first[n:]) and torch.equal(out[:n, :2], first[:n, :2])
        for ch, w in want.items():
            got = out[:n, 2:, ch]
            assert (torch.isnan(got) if w != w else got == w).all(), (places, ch, w)
        rest = torch.ones(128, dtype=torch.bool, device=DEV)
        rest[list(want)] = False
        assert torch.allclose(out[:n, 2:][..., rest], first[:n, 2:][..., rest], rtol=1e-5, atol=1e-6)


# ----------------------------------------------------------------- forms and layouts

@pytest.mark.parametrize("workspace", [True, False])
@pytest.mark.parametrize("lens,hq,hkv", [([(1, 3), (1, 7), (1, 40)], 4, 4), ([(2, 5), (1, 900), (3, 30)], 5, 1),
                                         ([(1, 1500), (1, 6)], 16, 1)])
def test_weights_of_few_rows_have_16_bits(lens, hq, hkv, workspace):
    """A weight as two bf16 is off by half a step of the low one, 2^-8 of at most 2^-8
    of it; scores of small queries add little (the sums of their magnitudes are
    about 1)."""
    e = 2.0 ** -24
    c = Case(lens, hq, hkv, 128, 16, "bf16")
    c.q.mul_(0.125)
    out, lse = _attend_into(c, c.q, workspace)
    ref, rl, mean, size = c.reference()
    bound = (2.0 ** -16 + 2 * (128 + 4) * e * size[..., None] + (c.max_kv + 64) * e) * mean
    err = np.abs(out.double().cpu().numpy() - ref)
    say(f"  few rows {lens}: of the bound {np.max(err / bound):.2f}, of one of 8 bits {np.max(err / mean) * 256:.4f}")
    assert np.all(err <= bound)


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
@pytest.mark.parametrize("lens", [[(1, 1), (1, 300)], [(1, 40), (1, 33), (1, 900)], [(2, 50), (0, 9), (1, 700), (9, 1400)]])
def test_more_query_heads_than_a_tile_has_rows(lens, cache):
    say(f"20 heads on one {lens} {cache}")
    c = Case(lens, 40, 2, 64, 16, cache)
    for workspace in (True, False):
        out, lse = _attend_into(c, c.q, workspace)
        c.check(out, lse, what="20 heads on one")


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_table_rows_further_apart_than_their_entries(cache):
    """The block table as some columns of a wider one, for the append and the attention."""
    say(f"wide table {cache}")
    lens = [(1, 70), (30, 130), (2, 2)]
    c, d = (Case(lens, 4, 2, 128, 32, cache, poison=False) for _ in range(2))
    wide = torch.full((3, c.table_d.shape[1] + 9), -5, dtype=torch.int32, device=DEV)
    wide[:, 4:4 + c.table_d.shape[1]] = c.table_d
    d.table_d = wide[:, 4:4 + c.table_d.shape[1]]
    c.append()
    d.append()
    out, lse = _attend_into(c, c.q, True)
    got, gl = _attend_into(d, d.q, True)
    assert torch.equal(got, out) and torch.equal(gl, lse)
    assert torch.equal(c.k.view(torch.uint8), d.k.view(torch.uint8)) and torch.equal(c.v.view(torch.uint8), d.v.view(torch.uint8))
    d.check(got, gl, what="wide table")


def test_one_token_has_no_stride():
    """The stride of a dimension of one says nothing: a single row of a wider or overlapping array is taken as it is."""
    c = Case([(1, 50)], 4, 2, 64, 16, "bf16")
    ref, rl = _attend_into(c, c.q, True)
    for step in (1, 4 * 64 + 1, 4 * 64 - 8, 4 * 64 + 8):
        q = c.q.contiguous().as_strided((1, 4, 64), (step, 64, 1))
        out, lse = _attend_into(c, q, True)
        assert torch.equal(out, ref) and torch.equal(lse, rl)
        k, v = (x.contiguous().as_strided((1, 2, 64), (step, 64, 1)) for x in (c.new_k, c.new_v))
        tb.tb_paged_append(k, v, c.k, c.v, c.table_d, c.cu_d, c.kv_d, c.max_q)
        torch.cuda.synchronize()
        i, s = int(c.table[0, 49 // 16]), 49 % 16
        assert torch.equal(c.k[i, :, s], c.new_k[0]) and torch.equal(c.v[i, :, :, s], c.new_v[0])
        ref, rl = _attend_into(c, c.q, True)


def test_table_of_one_column_has_no_stride():
    """Short sequences have a page each: their table is a row turned into a column."""
    c = Case([(1, 5), (2, 16), (1, 9)], 4, 2, 64, 16, "bf16")
    ref, rl = _attend_into(c, c.q, True)
    c.table_d = c.table_d[:, 0].contiguous()[None].t()
    assert c.table_d.stride() == (1, 3)
    out, lse = _attend_into(c, c.q, True)
    assert torch.equal(out, ref) and torch.equal(lse, rl)
    c.append()

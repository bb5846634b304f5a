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

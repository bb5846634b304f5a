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

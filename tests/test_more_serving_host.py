"""CPU tests of the rotary append, the 4-bit cache, its reader and the token
probabilities: refusals before any GPU work, in the C ABI and in the binding,
and the frequencies."""

import math
import os

import pytest
import torch

from ternary_weights_hadamard_amd import tb

built = pytest.mark.skipif(not os.path.exists(tb.LIB_PATH), reason="libtb.so not built")
pytestmark = built

A, B, C, D, E, F, G, H, I, J = (0x10000000 * i for i in range(1, 11))  # fake device addresses, never dereferenced
NULL, SHAPE, ALIGN, DTYPE, FORMAT, ALIAS, WORKSPACE, VALUE = 1, 2, 3, 4, 5, 8, 9, 10
F32, BF16, ACT8, FP8, INT4 = tb.TB_F32, tb.TB_BF16, tb.TB_ACT8, tb.TB_FP8, tb.TB_INT4


def _cache(**kw):
    a = dict(k_cache=A, v_cache=B, k_scale=I, v_scale=J, block_table=C, cu_q=D, kv_len=D + 4096, n_pages=8,
             table_stride=4, table_width=4, B=2, total_q=6, max_q=4, cache_dtype=INT4, page=16, heads_kv=2, head_dim=128)
    a.update(kw)
    return tb.PagedCache(**a)


def _rotary(cache=None, **kw):
    a = dict(cache=_cache(**(cache or {})), q=E, k=F, v=G, q_out=H, inv_freq=D + 8192, q_stride=1024, k_stride=256,
             v_stride=256, heads_q=8, rotary_dim=128, neighbours=0, turn_in=0, turn_out=0, turn_v=0, factor=1.0, reserved=0)
    a.update(kw)
    return tb.lib().tb_paged_append_rotary(tb.PagedRotaryArgs(**a), None)


def _append(**kw):
    return tb.lib().tb_paged_append(_cache(**kw), E, 256, F, 256, None)


def _attend(cache=None, **kw):
    a = dict(cache=_cache(**(cache or {})), q=E, out=F, lse=G, workspace=H, workspace_bytes=1 << 20, q_stride=1024,
             max_kv=64, window=0, heads_q=8, out_dtype=BF16, scale=1.0, reserved=0)
    a.update(kw)
    return tb.lib().tb_paged_attention(tb.PagedAttentionArgs(**a), None)


def _read(k=E, v=F, dtype=F32, **kw):
    return tb.lib().tb_paged_read(_cache(**kw), k, v, dtype, None)


CACHE_REFUSALS = [
    (DTYPE, dict(cache_dtype=5)), (DTYPE, dict(cache_dtype=ACT8)), (SHAPE, dict(head_dim=96)), (SHAPE, dict(page=8)),
    (SHAPE, dict(B=-1)), (SHAPE, dict(heads_kv=0)), (SHAPE, dict(table_width=5)), (SHAPE, dict(max_q=-1)),
    (NULL, dict(k_cache=None)), (NULL, dict(block_table=None)), (NULL, dict(kv_len=None)),
    (NULL, dict(k_scale=None)), (NULL, dict(v_scale=None)),
    (ALIGN, dict(k_scale=I + 4)), (ALIGN, dict(v_scale=J + 8)), (ALIGN, dict(v_cache=B + 4)), (ALIGN, dict(cu_q=D + 2)),
    (0, dict(B=0, cu_q=None)), (0, dict(total_q=0)), (0, dict(max_q=0)),
]


@pytest.mark.parametrize("status,kw", CACHE_REFUSALS)
def test_cache_refusals(status, kw):
    assert _append(**kw) == status
    assert _attend(cache=kw) == status
    assert _rotary(cache=kw) == status
    assert _read(**kw) == status


def test_scales_of_four_bits_are_part_of_the_cache():
    pool = 8 * 2 * 16 * 4   # bytes of the scales: 4 a position and head
    assert _append(k_scale=E + pool) == ALIAS                          # k of 6 tokens reaches there
    assert _append(k_scale=J) == ALIAS and _append(v_scale=A + 16) == ALIAS and _append(k_scale=C) == ALIAS
    assert _attend(out=I + pool - 16) == ALIAS and _attend(lse=J) == ALIAS
    assert _read(k=I + pool - 16) == ALIAS and _read(v=J) == ALIAS
    assert _rotary(q_out=I) == ALIAS and _rotary(cache=dict(v_scale=F)) == ALIAS
    # an 8-bit cache reads its scales, which are few: they may lie anywhere but in an output
    assert _read(k=I, cache_dtype=FP8) == ALIAS


@pytest.mark.parametrize("status,kw", [
    (SHAPE, dict(heads_q=0)), (SHAPE, dict(heads_q=70000, q_stride=1 << 24)), (SHAPE, dict(q_stride=1016)),
    (SHAPE, dict(q_stride=1028)), (SHAPE, dict(k_stride=128)), (SHAPE, dict(v_stride=260)), (SHAPE, dict(rotary_dim=-16)),
    (SHAPE, dict(rotary_dim=144)), (SHAPE, dict(rotary_dim=24)), (SHAPE, dict(reserved=1)),
    (SHAPE, dict(turn_in=1, cache=dict(head_dim=64))), (SHAPE, dict(turn_v=1, cache=dict(head_dim=64))),
    (SHAPE, dict(rotary_dim=80, cache=dict(head_dim=64))), (VALUE, dict(factor=math.nan)), (VALUE, dict(factor=math.inf)),
    (NULL, dict(k=None)), (NULL, dict(v=None)), (NULL, dict(q_out=None)), (NULL, dict(inv_freq=None)),
    (ALIGN, dict(q=E + 8)), (ALIGN, dict(q_out=H + 2)), (ALIGN, dict(k=F + 4)), (ALIGN, dict(inv_freq=D + 8194)),
    (ALIAS, dict(q_out=E)), (ALIAS, dict(q_out=A)), (ALIAS, dict(q_out=F)), (ALIAS, dict(k=A)), (ALIAS, dict(v=B + 512)),
    (ALIAS, dict(inv_freq=H + 64)), (ALIAS, dict(q_out=D)),
    # no queries, and no place for a key: nothing is done
    (0, dict(q=None, cache=dict(n_pages=0, k_cache=None, v_cache=None, k_scale=None, v_scale=None))),
    (0, dict(q=None, q_out=None, heads_q=0, q_stride=0, cache=dict(total_q=0))),
])
def test_rotary_refusals(status, kw):
    assert _rotary(**kw) == status


def test_read_refusals():
    assert tb.lib().tb_paged_read(None, E, F, F32, None) == NULL and tb.lib().tb_paged_append_rotary(None, None) == NULL
    assert _read(dtype=FP8) == DTYPE and _read(k=E + 8) == ALIGN and _read(v=F + 2) == ALIGN
    assert _read(v=E) == ALIAS and _read(k=A) == ALIAS and _read(v=C) == ALIAS
    assert _read(k=None, v=None) == 0 and _read(n_pages=0, k_cache=None) == 0


def _probs(**kw):
    a = dict(logits=A, p=B, params=C, drafts=D, cu_draft=D + 4096, history=E, cu_history=E + (1 << 20), prompt_len=E + (1 << 21),
             bias_ids=F, bias_values=F + (1 << 20), cu_bias=F + (1 << 21), mask=G, mask_row=G + (1 << 20), workspace=H,
             workspace_bytes=1 << 20, B=2, total=6, vocab=1000, logits_stride=1000, p_stride=1000, total_history=100,
             total_bias=10, n_masks=3, mask_stride=32, max_draft=4, logits_dtype=F32, p_dtype=F32, reserved=0)
    a.update(kw)
    return tb.lib().tb_token_probs(tb.TokenProbsArgs(**a), None)


BIG = dict(vocab=300000, logits_stride=300000, p_stride=300000, mask_stride=10000)


@pytest.mark.parametrize("status,kw", [
    (DTYPE, dict(logits_dtype=ACT8)), (DTYPE, dict(p_dtype=FP8)), (SHAPE, dict(B=-1)), (SHAPE, dict(B=65536)),
    (SHAPE, dict(total=-1)), (SHAPE, dict(vocab=0)), (SHAPE, dict(max_draft=-1)), (SHAPE, dict(max_draft=65)),
    (SHAPE, dict(logits_stride=999)), (SHAPE, dict(p_stride=999)), (SHAPE, dict(reserved=2)), (SHAPE, dict(total_history=-1)),
    (SHAPE, dict(total_bias=-1)), (SHAPE, dict(n_masks=-1)), (SHAPE, dict(mask_stride=31)),
    (SHAPE, dict(mask_row=None)),                               # three masks for eight rows
    (NULL, dict(logits=None)), (NULL, dict(p=None)), (NULL, dict(params=None)), (NULL, dict(drafts=None)),
    (NULL, dict(cu_draft=None)), (NULL, dict(cu_history=None)), (NULL, dict(bias_values=None)), (NULL, dict(cu_bias=None)),
    (ALIGN, dict(logits=A + 2)), (ALIGN, dict(p=B + 1, p_dtype=BF16)), (ALIGN, dict(params=C + 8)),
    (ALIGN, dict(history=E + 2)), (ALIGN, dict(mask=G + 2)), (ALIGN, dict(workspace=H + 4)),
    (WORKSPACE, dict(workspace=None, **BIG)), (WORKSPACE, dict(workspace_bytes=16, **BIG)),
    (ALIAS, dict(p=A)), (ALIAS, dict(p=C)), (ALIAS, dict(p=E)), (ALIAS, dict(p=G + 64)), (ALIAS, dict(p=D + 4096)),
    (ALIAS, dict(workspace=A, **BIG)), (ALIAS, dict(workspace=B + 4096, **BIG)),
    (0, dict(B=0, total=0, logits=None)),
])
def test_probs_refusals(status, kw):
    assert _probs(**kw) == status


def test_probs_workspace():
    def ws(**kw):
        a = dict(B=2, total=6, vocab=1 << 15, logits_stride=1 << 20, p_stride=1 << 20, max_draft=4, logits_dtype=F32,
                 p_dtype=F32)
        a.update(kw)
        return tb.lib().tb_token_probs_workspace(tb.TokenProbsArgs(**a))

    assert ws() == 0 and ws(B=0, total=0) == 0 and ws(vocab=-1) == 0 and tb.lib().tb_token_probs_workspace(None) == 0
    one = ws(vocab=(1 << 15) + 1)
    assert one > 0 and ws(vocab=(1 << 15) + 1, total=14) == 2 * one


def test_frequencies():
    f, m = tb.tb_rotary_frequencies(64, base=500000.0)
    want = torch.tensor([500000.0 ** (-2 * i / 64) for i in range(32)], dtype=torch.float64).float()
    assert m == 1.0 and torch.equal(f, want)
    f, m = tb.tb_rotary_frequencies(64, base=500000.0, scaling=tb.TB_ROPE_LINEAR, scale=4.0)
    assert m == 1.0 and torch.equal(f, (want.double() / 4).float())
    # the slowest pair turns as far over the longer context as it did, the fastest stays
    f, m = tb.tb_rotary_frequencies(64, base=10000.0, scaling=tb.TB_ROPE_NTK, scale=8.0)
    p, _ = tb.tb_rotary_frequencies(64, base=10000.0)
    assert m == 1.0 and f[0] == 1.0 and abs(f[31] / p[31] * 8 - 1) < 1e-6 and (f[1:31] < p[1:31]).all()
    f, m = tb.tb_rotary_frequencies(128, base=10000.0, scaling=tb.TB_ROPE_YARN, scale=4.0, trained=4096)
    p, _ = tb.tb_rotary_frequencies(128, base=10000.0)
    c = lambda n: 128 * math.log(4096 / (2 * math.pi * n)) / (2 * math.log(10000.0))  # noqa: E731
    lo, hi = math.floor(c(32)), math.ceil(c(1))
    assert 0 < lo < hi < 64 and abs(m - (0.1 * math.log(4) + 1)) < 1e-7
    assert torch.equal(f[:lo + 1], p[:lo + 1]) and torch.allclose(f[hi:], p[hi:] / 4, rtol=2.0 ** -23)
    r = (torch.arange(64).double() - lo) / (hi - lo)
    mid = slice(lo, hi + 1)
    assert torch.allclose(f[mid].double(), p[mid].double() * (1 - r[mid] + r[mid] / 4), rtol=2.0 ** -22)


@pytest.mark.parametrize("code,kw", [
    (SHAPE, dict(rotary_dim=0)), (SHAPE, dict(rotary_dim=24)), (SHAPE, dict(rotary_dim=144)), (FORMAT, dict(scaling=4)),
    (VALUE, dict(base=1.0)), (VALUE, dict(base=math.inf)), (VALUE, dict(scale=0.5)), (VALUE, dict(scale=math.nan)),
    (VALUE, dict(scaling=tb.TB_ROPE_YARN)), (VALUE, dict(scaling=tb.TB_ROPE_YARN, trained=4096, fast=0.0)),
    (VALUE, dict(scaling=tb.TB_ROPE_YARN, trained=4096, slow=math.inf)),
    (VALUE, dict(scaling=tb.TB_ROPE_NTK, base=1e300, scale=1e300)),
])
def test_frequencies_refused(code, kw):
    kw = dict(dict(rotary_dim=64), **kw)
    with pytest.raises(tb.TBError) as e:
        tb.tb_rotary_frequencies(**kw)
    assert e.value.code == code
    assert tb.lib().tb_rotary_frequencies(64, 10000.0, 0, 1.0, 0.0, 1.0, 1.0, None, None) == NULL


def test_binding_refuses():
    i = torch.zeros(2, dtype=torch.int32)
    kc, vc = torch.zeros(2, 1, 16, 64, dtype=torch.uint8), torch.zeros(2, 1, 64, 16, dtype=torch.uint8)
    q = torch.zeros(1, 1, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        tb.tb_paged_append_rotary(q, q, q, kc, vc, i[None], i, i[:1], 1, None)
    with pytest.raises(ValueError):
        tb.tb_paged_read(kc, vc, i[None], i, i[:1], 1, 1)
    with pytest.raises(ValueError):
        tb.tb_token_probs(torch.zeros(1, 8), torch.zeros(1, 4))

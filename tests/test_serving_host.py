"""CPU tests of the serving operators: refusals before any GPU work, in the C
ABI and in the binding, and the cache's bounds on wrong entries."""

import ctypes
import os
import shutil
import subprocess

import pytest
import torch

from ternary_weights_hadamard_amd import tb

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

built = pytest.mark.skipif(not os.path.exists(tb.LIB_PATH), reason="libtb.so not built")

A, B, C, D, E, F, G, H = (0x1000000 * i for i in range(1, 9))  # fake device addresses, never dereferenced
NULL, SHAPE, ALIGN, DTYPE, ALIAS, WORKSPACE, VALUE = 1, 2, 3, 4, 8, 9, 10
F32, BF16, ACT8, FP8 = tb.TB_F32, tb.TB_BF16, tb.TB_ACT8, tb.TB_FP8


def _norm(**kw):
    a = dict(y=A, resid=B, w_post=C, w_pre=D, gate=E, h=F, z=G, rows=4, C=256, rows_per_gate=1, parts=1, y_dtype=BF16,
             h_dtype=BF16, w_dtype=BF16, gate_dtype=BF16, z_dtype=BF16, rotate_in=0, rotate_out=0, alpha=1.0, eps=1e-6)
    a.update(kw)
    return tb.lib().tb_block_norm(tb.BlockNormArgs(**a), None)


@built
@pytest.mark.parametrize("status,kw", [
    (SHAPE, dict(C=200)), (SHAPE, dict(C=0)), (SHAPE, dict(C=tb.TB_NORM_MAX_C + 128)), (SHAPE, dict(rows=-1)),
    (SHAPE, dict(parts=9, y_dtype=F32)), (SHAPE, dict(parts=-1)), (SHAPE, dict(rows_per_gate=0)),
    (DTYPE, dict(parts=2)), (DTYPE, dict(y_dtype=ACT8)), (DTYPE, dict(h_dtype=ACT8)), (DTYPE, dict(z_dtype=FP8)),
    (DTYPE, dict(w_dtype=9)), (DTYPE, dict(gate_dtype=-1)),
    (VALUE, dict(eps=0.0)), (VALUE, dict(eps=float("nan"))), (VALUE, dict(alpha=float("inf"))),
    (NULL, dict(h=None, z=None)), (NULL, dict(y=None, resid=None)), (NULL, dict(w_pre=None)),
    (ALIGN, dict(y=A + 8)), (ALIGN, dict(gate=E + 4)), (ALIGN, dict(z=G + 2)),
    (ALIAS, dict(h=A)), (ALIAS, dict(z=B)), (ALIAS, dict(z=F)), (ALIAS, dict(h=B + 16)), (ALIAS, dict(z=C + 256)),
    (ALIAS, dict(z=A - 4 * 256 * 4, z_dtype=ACT8)),   # 4 rows of the operand reach past 4 fp32 rows
    (ALIAS, dict(parts=4, y_dtype=F32, z=A + 3 * 4 * 256 * 4)),
    (0, dict(rows=0, y=None, resid=None, h=None, z=None)),
])
def test_block_norm_refusals(status, kw):
    assert _norm(**kw) == status


def _cache(**kw):
    a = dict(k_cache=A, v_cache=B, k_scale=None, v_scale=None, block_table=C, cu_q=D, kv_len=D + 4096, n_pages=8,
             table_stride=4, table_width=4, B=2, total_q=6, max_q=4, cache_dtype=BF16, page=16, heads_kv=2, head_dim=128)
    a.update(kw)
    return tb.PagedCache(**a)


def _append(k=E, ks=256, v=F, vs=256, **kw):
    return tb.lib().tb_paged_append(_cache(**kw), k, ks, v, vs, None)


def _attend(cache=None, **kw):
    a = dict(cache=_cache(**(cache or {})), q=E, out=F, lse=G, workspace=H, workspace_bytes=1 << 20, q_stride=1024,
             max_kv=64, window=0, heads_q=8, out_dtype=BF16, scale=1.0, reserved=0)
    a.update(kw)
    return tb.lib().tb_paged_attention(tb.PagedAttentionArgs(**a), None)


CACHE_REFUSALS = [
    (DTYPE, dict(cache_dtype=F32)), (SHAPE, dict(head_dim=96)), (SHAPE, dict(page=8)), (SHAPE, dict(page=48)),
    (SHAPE, dict(page=2048)), (SHAPE, dict(B=-1)), (SHAPE, dict(B=65536)), (SHAPE, dict(heads_kv=0)),
    (SHAPE, dict(n_pages=-1)), (SHAPE, dict(total_q=-1)), (SHAPE, dict(max_q=-1)), (SHAPE, dict(table_width=5)),
    (SHAPE, dict(table_width=-1)), (SHAPE, dict(table_width=(1 << 26) + 1, table_stride=1 << 27)), (SHAPE, dict(total_q=(1 << 27) + 1)),
    (NULL, dict(k_cache=None)), (NULL, dict(v_cache=None)), (NULL, dict(block_table=None)), (NULL, dict(cu_q=None)),
    (NULL, dict(kv_len=None)), (ALIGN, dict(k_cache=A + 8)), (ALIGN, dict(v_cache=B + 2)), (ALIGN, dict(cu_q=D + 1)),
    (ALIGN, dict(block_table=C + 2)), (ALIGN, dict(kv_len=D + 4098)), (ALIGN, dict(k_scale=G + 2)),
    (0, dict(B=0, cu_q=None)), (0, dict(total_q=0)), (0, dict(max_q=0)),
]


@built
@pytest.mark.parametrize("status,kw", CACHE_REFUSALS)
def test_cache_refusals(status, kw):
    assert _append(**kw) == status
    assert _attend(cache=kw) == status


@built
def test_append_refusals():
    assert tb.lib().tb_paged_append(None, E, 256, F, 256, None) == NULL
    assert _append(k=None) == NULL and _append(v=None) == NULL
    assert _append(k=E + 8) == ALIGN
    assert _append(ks=255) == SHAPE and _append(vs=260) == SHAPE and _append(ks=128) == SHAPE
    assert _append(v_cache=A) == ALIAS                       # one pool for both
    assert _append(k=A + 4096) == ALIAS and _append(v=B) == ALIAS and _append(block_table=A) == ALIAS
    assert _append(n_pages=0, k_cache=None, v_cache=None) == 0  # nowhere to write
    assert _append(table_width=0, block_table=None) == 0


@built
def test_attention_refusals():
    assert tb.lib().tb_paged_attention(None, None) == NULL
    assert _attend(q=None) == NULL and _attend(out=None) == NULL
    assert _attend(q=E + 2) == ALIGN and _attend(out=F + 8) == ALIGN and _attend(lse=G + 2) == ALIGN
    assert _attend(workspace=H + 8) == ALIGN
    assert _attend(heads_q=7) == SHAPE and _attend(heads_q=0) == SHAPE
    assert _attend(q_stride=1016) == SHAPE and _attend(q_stride=1028) == SHAPE
    assert _attend(window=-1) == SHAPE and _attend(max_kv=-1) == SHAPE and _attend(reserved=1) == SHAPE
    assert _attend(out_dtype=ACT8) == DTYPE
    assert _attend(scale=float("nan")) == VALUE
    assert _attend(cache=dict(max_q=1 << 25, total_q=1 << 25)) == SHAPE    # more rows than a launch takes
    assert _attend(out=E) == ALIAS and _attend(out=A + 16) == ALIAS and _attend(lse=F) == ALIAS
    assert _attend(out=D) == ALIAS and _attend(lse=C) == ALIAS


@built
def test_attention_workspace():
    def ws(cache=None, **kw):
        a = dict(cache=_cache(**(cache or {})), q_stride=1024, max_kv=64, window=0, heads_q=8, out_dtype=BF16, scale=1.0)
        a.update(kw)
        return tb.lib().tb_paged_attention_workspace(tb.PagedAttentionArgs(**a))

    assert ws() == 0                                         # short: one part
    row = (128 + 2) * 4                                      # values and two statistics
    long = ws(max_kv=1 << 16)
    assert long > 0 and long % row == 0
    assert ws(max_kv=1 << 16, window=64) <= long
    assert ws(max_kv=1 << 16, heads_q=7) == 0 and ws(cache=dict(B=0), max_kv=1 << 16) == 0
    # what the call would write is the workspace it is checked against
    assert _attend(max_kv=1 << 16, workspace=F, workspace_bytes=long) == ALIAS


def _verify(**kw):
    a = dict(p=A, q=B, drafts=C, u=C + 4096, u_next=C + 8192, cu_draft=C + 12288, accepted=D, tokens=D + 4096, workspace=E,
             workspace_bytes=1 << 20, B=2, total=6, vocab=1000, p_stride=1000, q_stride=1000, max_draft=4, p_dtype=F32,
             q_dtype=F32, reserved=0)
    a.update(kw)
    return tb.lib().tb_verify_draft(tb.VerifyDraftArgs(**a), None)


BIG = dict(vocab=300000, p_stride=300000, q_stride=300000)


@built
@pytest.mark.parametrize("status,kw", [
    (DTYPE, dict(p_dtype=ACT8)), (DTYPE, dict(q_dtype=7)), (SHAPE, dict(B=-1)), (SHAPE, dict(B=65536)),
    (SHAPE, dict(total=-1)), (SHAPE, dict(vocab=0)), (SHAPE, dict(max_draft=-1)), (SHAPE, dict(max_draft=65)),
    (SHAPE, dict(p_stride=999)), (SHAPE, dict(q_stride=999)), (SHAPE, dict(reserved=2)),
    (NULL, dict(p=None)), (NULL, dict(u=None)), (NULL, dict(u_next=None)), (NULL, dict(drafts=None)),
    (NULL, dict(cu_draft=None)), (NULL, dict(accepted=None)), (NULL, dict(tokens=None)),
    (ALIGN, dict(p=A + 2)), (ALIGN, dict(q=B + 1, q_dtype=BF16)), (ALIGN, dict(u=C + 4098)), (ALIGN, dict(workspace=E + 4)),
    (WORKSPACE, dict(workspace=None, **BIG)), (WORKSPACE, dict(workspace_bytes=16, **BIG)),
    (ALIAS, dict(tokens=D)), (ALIAS, dict(accepted=C)), (ALIAS, dict(workspace=A, **BIG)), (ALIAS, dict(tokens=B + 400)),
    (0, dict(B=0, p=None)),
])
def test_verify_refusals(status, kw):
    assert _verify(**kw) == status


@built
def test_verify_workspace():
    assert tb.tb_verify_draft_workspace(0, 100) == 0 and tb.tb_verify_draft_workspace(1, 0) == 0
    assert tb.tb_verify_draft_workspace(3, 1 << 15) == 0 and tb.tb_verify_draft_workspace(3, (1 << 15) + 1) > 0


@built
def test_binding_refuses():
    """Tensors that are not on the device, or of the wrong shape, are refused before the library is called."""
    t = torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        tb.tb_block_norm(t, t, w_pre=t[0])
    with pytest.raises(ValueError):
        tb.tb_block_norm(None)
    i = torch.zeros(2, dtype=torch.int32)
    kc, vc = torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16), torch.zeros(2, 1, 64, 16, dtype=torch.bfloat16)
    q = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        tb.tb_paged_append(q, q, kc, vc, i[None], i, i[:1], 1)
    with pytest.raises(ValueError):
        tb.tb_paged_attention(q, kc, vc, i[None], i, i[:1], 1, 16)
    f = torch.zeros(1)
    with pytest.raises(ValueError):
        tb.tb_verify_draft(torch.zeros(2, 8), torch.zeros(1, 8), i[:1], f, f, i, 1)


PROBE = r"""
#include "paged.h"
extern "C" void probe(const int32_t* cu, const int32_t* kv, int64_t b, int64_t total, int64_t cap, int64_t j0, int64_t j1,
                      int64_t window, int64_t* out) {
  tb::PagedSeq s = tb::paged_seq(cu, kv, b, total, cap);
  tb::PagedSpan r = tb::paged_span(s, (int)j0, (int)j1, window);
  int64_t v[6] = {s.row0, s.n, s.keys, s.first_pos, r.begin, r.end};
  for (int i = 0; i < 6; ++i) out[i] = v[i];
}
extern "C" int page(const int32_t* row, int64_t width, int64_t pages, int64_t i) { return tb::paged_page(row, width, pages, i); }
"""


@pytest.mark.skipif(shutil.which("g++") is None, reason="no host compiler")
def test_cache_bounds_on_wrong_entries(tmp_path):
    """The functions through which the kernels reach the cache, compiled for the
    host: no entry of cu_q, kv_len or block_table leads outside the arrays."""
    src, so = tmp_path / "probe.cpp", tmp_path / "probe.so"
    src.write_text(PROBE)
    csrc = os.path.join(ROOT, "ternary_weights_hadamard_amd", "csrc")
    subprocess.run(["g++", "-O1", "-shared", "-fPIC", f"-I{csrc}", str(src), "-o", str(so)], check=True)
    L = ctypes.CDLL(str(so))
    i32, i64 = ctypes.c_int32, ctypes.c_int64

    def seq(cu, kv, total=10, cap=64, j0=0, j1=0, window=0):
        out = (i64 * 6)()
        L.probe((i32 * 2)(*cu), (i32 * 1)(kv), i64(0), i64(total), i64(cap), i64(j0), i64(j1), i64(window), out)
        return list(out)

    assert seq((2, 5), 20, j1=2) == [2, 3, 20, 17, 0, 20]
    assert seq((2, 5), 20, j1=1, window=4) == [2, 3, 20, 17, 14, 19]
    assert seq((-3, 5), 20)[:2] == [0, 5]
    assert seq((4, 99), 20)[:2] == [4, 6]
    assert seq((7, 2), 20)[:2] == [7, 0]
    assert seq((50, 60), 20)[:2] == [10, 0]
    assert seq((0, 1), -5, j1=0) == [0, 1, 0, -1, 0, 0]
    assert seq((0, 1), 2**31 - 1, j1=0) == [0, 1, 64, 2**31 - 2, 0, 64]       # no further than the table
    assert seq((0, 1), 2**31 - 1, j1=0, window=5)[4:] == [64, 64]
    assert seq((0, 1), 20, j1=0, window=2**31 - 1)[4:] == [0, 20]
    assert seq((0, 5), 2, j1=4) == [0, 5, 2, -3, 0, 2]
    assert seq((0, 5), 2, j1=1)[4:] == [0, 0]                                  # tokens before position 0
    row = (i32 * 4)(3, -1, 8, -2**31)
    got = [L.page(row, i64(4), i64(8), i64(i)) for i in (-1, 0, 1, 2, 3, 4, 2**40)]
    assert got == [-1, 3, -1, -1, -1, -1, -1]

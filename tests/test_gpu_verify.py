"""GPU results of tb_verify_draft against the oracle.  Whole numbers, so equal:
the probabilities of the exact cases are multiples of 2^-k whose sums have no
rounding, edges (u q = p, a draw on a weight's end) among them; those of the
others are random, where 64-bit sums in another order move an edge by 1e-16."""

import numpy as np
import pytest
import torch

import oracle
from gpu_util import DEV, say
from ternary_weights_hadamard_amd import tb

pytestmark = pytest.mark.gpu


def _dev(a, dtype=torch.float32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(dtype).to(DEV)


def _run(p, q, drafts, u, u_next, cu, max_draft, pk=torch.float32, qk=torch.float32, **kw):
    pd, qd = _dev(p, pk), None if q is None else _dev(q, qk)
    acc, tok = tb.tb_verify_draft(pd, qd, _dev(drafts, torch.int32), _dev(u), _dev(u_next), _dev(cu, torch.int32),
                                  max_draft, **kw)
    torch.cuda.synchronize()
    pv = pd.double().cpu().numpy()
    qv = None if qd is None else qd.double().cpu().numpy()
    u32 = lambda a: np.asarray(a, np.float32).astype(np.float64)  # noqa: E731
    ra, rt = oracle.serving.verify_draft(pv, qv, drafts, u32(u), u32(u_next), cu, max_draft)
    assert np.array_equal(acc.cpu().numpy(), ra), (acc.tolist(), ra.tolist())
    assert np.array_equal(tok.cpu().numpy(), rt), (tok.tolist(), rt.tolist())
    return ra, rt


def _dyadic(rng, rows, vocab, zeros=0.3):
    """Rows of multiples of 2^-10 (exact in bf16 too: below 2^8 of them), many 0."""
    c = rng.integers(1, 200, (rows, vocab)) * (rng.random((rows, vocab)) > zeros)
    c[:, 0] += c.sum(1) == 0
    return c / 1024.0


def _ragged(rng, b, t):
    n = rng.integers(0, t + 1, b)
    n[0] = t
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int64)


@pytest.mark.parametrize("vocab", [1, 2, 63, 64, 65, 2047, 2048, 2049, 4095, 4097, 4100, 32003, 32768, 32769, 262145])
@pytest.mark.parametrize("kind", ["dense", "certain"])
def test_verify_exact_weights(vocab, kind):
    say(f"verify vocab {vocab} {kind}")
    rng = np.random.default_rng(vocab)
    b, t = 9, 5
    cu = _ragged(rng, b, t)
    total = int(cu[-1])
    p, q = _dyadic(rng, total + b, vocab), _dyadic(rng, total, vocab)
    drafts = rng.integers(0, vocab, total)
    u = rng.integers(0, 8, total) / 8.0
    _run(p, q if kind == "dense" else None, drafts, u, rng.integers(0, 16, b) / 16.0, cu, t)
    # drafts that are mostly kept: q is p / 2
    half = np.concatenate([p[cu[i] + i:cu[i + 1] + i] for i in range(b)]) / 2
    acc, _ = _run(p, half, drafts, u, rng.integers(0, 16, b) / 16.0, cu, t)
    _run(p, q if kind == "dense" else None, drafts, u, np.zeros(b), cu, t, pk=torch.bfloat16, qk=torch.bfloat16)


@pytest.mark.parametrize("seed", range(4))
def test_verify_random(seed):
    rng = np.random.default_rng(seed)
    b, t, vocab = 6, 8, 5003
    cu = _ragged(rng, b, t)
    total = int(cu[-1])
    x = rng.standard_normal((total + b, vocab)) * 3
    p = np.exp(x) / np.exp(x).sum(1, keepdims=True)
    own = np.concatenate([np.arange(cu[i] + i, cu[i + 1] + i) for i in range(b)])
    y = x[own] + 0.3 * rng.standard_normal((total, vocab))
    q = np.exp(y) / np.exp(y).sum(1, keepdims=True)
    drafts = np.array([rng.choice(vocab, p=r / r.sum()) for r in q])
    for pk, qk in ((torch.float32, torch.float32), (torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)):
        acc, _ = _run(p, q, drafts, rng.random(total), rng.random(b), cu, t, pk, qk)
    say("accepted", acc.tolist())


def test_verify_edges():
    v = 300
    p = np.zeros((3, v))
    p[0, 7], p[0, 200] = 0.25, 0.75
    p[1, 5] = 1.0
    q = np.zeros((1, v))
    q[0, 7] = 0.5
    cu = [0, 1, 1]
    # u q = p is not kept; what is left is token 200.  Sequence 1 draws from p[2], which holds nothing
    assert _run(p, q, [7], [0.5], [0.0, 0.999], cu, 1)[1].tolist() == [[200, -1], [-1, -1]]
    assert _run(p, q, [7], [0.49], [0.0, 0.0], cu, 1)[1].tolist() == [[7, 5], [-1, -1]]
    # p = q with a draft of no probability: nothing is left, p itself
    assert _run(p, p[:1], [9], [0.0], [0.3, 0.0], cu, 1)[1].tolist() == [[200, -1], [-1, -1]]
    # a row without a positive finite weight draws nothing
    p2 = np.zeros((1, v))
    p2[0, :4] = [np.nan, np.inf, -1.0, 0.0]
    assert _run(p2, None, np.zeros(0, np.int64), np.zeros(0), [0.5], [0, 0], 0)[1].tolist() == [[-1]]
    # NaN in p or q is not kept and has no weight
    p3 = np.full((2, v), 0.25)
    p3[0, 7] = np.nan
    assert _run(p3, q, [7], [0.0], [0.0], [0, 1], 1)[0].tolist() == [0]
    q3 = q.copy()
    q3[0, 7] = np.nan
    assert _run(np.full((2, v), 0.25), q3, [7], [0.0], [0.0], [0, 1], 1)[0].tolist() == [0]


def test_verify_draft_ids_outside_the_vocabulary():
    p = np.full((3, 10), 0.125)
    q = np.full((2, 10), 0.0625)
    for bad in (-1, 10, 2**31 - 1, -2**31):
        assert _run(p, q, [3, bad], [0.5, 0.0], [0.5], [0, 2], 2)[0].tolist() == [1]
        assert _run(p, None, [bad, 3], [0.0, 0.0], [0.5], [0, 2], 2)[0].tolist() == [0]


def test_verify_long_drafts_and_max_draft():
    t, v = 64, 50
    p, q = np.full((t + 1, v), 1 / 64), np.full((t, v), 1 / 128)
    acc, tok = _run(p, q, np.arange(t) % v, np.full(t, 0.5), [0.0], [0, t], t)
    assert acc.tolist() == [64] and tok[0, -1] == 0
    # drafts past max_draft are not looked at
    pd, qd = _dev(p), _dev(q)
    acc, tok = tb.tb_verify_draft(pd, qd, _dev(np.arange(t) % v, torch.int32), _dev(np.full(t, 0.5)), _dev([0.0]),
                                  _dev([0, t], torch.int32), 3)
    torch.cuda.synchronize()
    assert acc.tolist() == [3] and tok.tolist() == [[0, 1, 2, 0]]


def test_verify_strides_alignment_and_given_outputs():
    rng = np.random.default_rng(5)
    b, t, v = 4, 3, 1001
    cu = _ragged(rng, b, t)
    total = int(cu[-1])
    p, q = _dyadic(rng, total + b, v), _dyadic(rng, total, v)
    drafts, u, un = rng.integers(0, v, total), rng.integers(0, 8, total) / 8, rng.integers(0, 8, b) / 8
    ra, rt = _run(p, q, drafts, u, un, cu, t)
    for kind in (torch.float32, torch.bfloat16):
        wide_p = torch.full((total + b, v + 7), float("nan"), device=DEV, dtype=kind)
        wide_q = torch.full((total, v + 3), float("nan"), device=DEV, dtype=kind)
        wide_p[:, 1:v + 1] = _dev(p, kind)
        wide_q[:, 3:v + 3] = _dev(q, kind)
        acc = torch.empty(b, dtype=torch.int32, device=DEV)
        tok = torch.empty(b, t + 1, dtype=torch.int32, device=DEV)
        rest = _dev(drafts, torch.int32), _dev(u), _dev(un), _dev(cu, torch.int32)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        got = tb.tb_verify_draft(wide_p[:, 1:v + 1], wide_q[:, 3:], *rest, t, accepted=acc, tokens=tok, stream=s)
        s.synchronize()
        assert got[0] is acc and got[1] is tok
        assert np.array_equal(acc.cpu().numpy(), ra) and np.array_equal(tok.cpu().numpy(), rt)


def test_verify_offsets_outside_the_arrays():
    """cu_draft that falls or leaves the arrays is clamped on the device: nothing outside them is read."""
    p, q = _dev(np.full((6, 40), 0.125)), _dev(np.full((3, 40), 0.0625))
    d, u, un = _dev([1, 2, 3], torch.int32), _dev([0.5, 0.5, 0.5]), _dev([0.0, 0.0, 0.0])
    for cu in ([-5, 1, 2, 99], [0, 3, 1, 2], [7, 8, 9, 10], [0, 2**31 - 1, -2**31, 3]):
        acc, tok = tb.tb_verify_draft(p, q, d, u, un, _dev(cu, torch.int32), 3)
        torch.cuda.synchronize()
        assert (acc >= 0).all() and (acc <= 3).all() and (tok < 40).all()


@pytest.mark.parametrize("v", [3001, 300001])
def test_verify_in_a_graph(v):
    rng = np.random.default_rng(8)
    b, t = 3, 4
    cu = np.arange(b + 1) * t
    p, q = _dev(_dyadic(rng, b * t + b, v)), _dev(_dyadic(rng, b * t, v))
    d, u, un = _dev(rng.integers(0, v, b * t), torch.int32), _dev(rng.random(b * t)), _dev(rng.random(b))
    cud = _dev(cu, torch.int32)
    acc, tok = torch.zeros(b, dtype=torch.int32, device=DEV), torch.zeros(b, t + 1, dtype=torch.int32, device=DEV)
    ws = torch.empty(max(tb.tb_verify_draft_workspace(b, v), 16), dtype=torch.uint8, device=DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tb.tb_verify_draft(p, q, d, u, un, cud, t, accepted=acc, tokens=tok, workspace=ws)
    for _ in range(4):
        u.uniform_()
        un.uniform_()
        d.random_(0, v)
        g.replay()
        torch.cuda.synchronize()
        ea, et = tb.tb_verify_draft(p, q, d, u, un, cud, t)
        assert torch.equal(acc, ea) and torch.equal(tok, et)

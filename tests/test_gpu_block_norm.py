"""GPU parity of tb_block_norm against the oracle.

Bounds: with e = 2^-24 (half an fp32 step), a row's sum of squares is off by at
most (8 + 6 + 16 + 4) e relative (lanes, wave, waves, the rest), which enters by
half; parts, gate, weight, residual and rsqrt add fewer than 40 e of the row's
largest terms: 64 e of their sum.  A rotation adds up to 7 e of a block's
absolute sum, at most 128 / sqrt(128) of its largest element.  z inherits h's.
A bf16 output adds half a step, 2^-8 relative.
"""

import numpy as np
import pytest
import torch

import oracle
from gpu_util import DEV, act8_decode, act8_kept, host_f64, say
from ternary_weights_hadamard_amd import tb

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
KIND = {"f32": torch.float32, "bf16": torch.bfloat16}


def _t(rng, shape, kind, scale=1.0, shift=0.0):
    x = torch.from_numpy((rng.standard_normal(shape) * scale + shift).astype(np.float32))
    return x.to(KIND[kind]).to(DEV)


def _check(got, ref, terms, rotated, what):
    """|got - ref| within the bounds above; `terms` is the largest magnitude of
    what a row's elements were summed from."""
    k = 64 * E * terms + (7 * 12 * E * terms * 12 if rotated else 0.0)
    half = np.abs(ref) * 2.0 ** -8 if got.dtype == torch.bfloat16 else 0.0
    err = np.abs(host_f64(got) - ref)
    say(f"  {what}: max err {err.max(initial=0):.3e}")
    assert np.all(np.isfinite(host_f64(got)))
    assert np.all(err <= k + half + 1e-30), what


CASES = [
    # rows, C, parts, y, stream, weights, gate (None or rows a gate serves), rotate in, out, z
    (1, 128, 1, "bf16", "bf16", "bf16", None, False, False, "bf16"),
    (1, 5120, 4, "f32", "f32", "bf16", None, True, True, "bf16"),
    (3, 5120, 8, "f32", "bf16", "f32", 1, True, True, "f32"),
    (17, 640, 1, "bf16", "f32", "f32", 5, True, False, "f32"),
    (7, 8192, 2, "f32", "bf16", "bf16", 7, False, True, "bf16"),
    (5, 8320, 1, "bf16", "bf16", "bf16", 2, False, True, "bf16"),
    (2, 17408, 1, "f32", "f32", "bf16", 1, True, True, "bf16"),
    (2, 32768, 3, "f32", "bf16", "f32", 2, True, True, "f32"),
    (333, 256, 1, "bf16", "bf16", "bf16", 1, False, False, "bf16"),
]


def _inputs(case, seed=0):
    rows, c, parts, yk, sk, wk, per, rin, rout, zk = case
    rng = np.random.default_rng(rows + c + seed)
    y = _t(rng, (parts, rows, c) if parts > 1 else (rows, c), yk)
    resid = _t(rng, (rows, c), sk, 2.0)
    w_post, w_pre = _t(rng, (c,), wk, 0.2, 1.0), _t(rng, (c,), wk, 0.2, 1.0)
    gate = None if per is None else _t(rng, (-(-rows // per), c), wk)
    return y, resid, w_post, w_pre, gate


def _ref(y, resid, w_post, w_pre, gate, per, alpha, eps, rin, rout):
    f = lambda t: None if t is None else host_f64(t)  # noqa: E731
    yy = f(y)
    if yy is not None and yy.ndim == 2:
        yy = yy[None]
    return oracle.serving.block_norm(yy, f(resid), f(w_post), f(w_pre), f(gate), per or 1, alpha, eps, rin, rout)


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_block_norm_matches_oracle(case):
    rows, c, parts, yk, sk, wk, per, rin, rout, zk = case
    say(f"block norm {case}")
    y, resid, w_post, w_pre, gate = _inputs(case)
    alpha, eps = 0.7, 1e-5
    h, z = tb.tb_block_norm(y, resid, w_post=w_post, w_pre=w_pre, gate=gate, rows_per_gate=per or 1, alpha=alpha, eps=eps,
                            y_parts=parts, rotate_in=rin, rotate_out=rout, z_dtype=KIND[zk])
    torch.cuda.synchronize()
    rh, rz = _ref(y, resid, w_post, w_pre, gate, per, alpha, eps, rin, rout)
    terms = np.abs(rh).max() + np.abs(host_f64(resid)).max() + 2 * parts * np.abs(host_f64(y)).max()
    assert h.dtype == resid.dtype and z.dtype == KIND[zk]
    _check(h, rh, terms, rin, "h")
    _check(z, rz, 4 * max(terms, np.abs(rz).max()), rin or rout, "z")


def test_block_norm_optional_arguments():
    case = (5, 384, 1, "bf16", "bf16", "bf16", 5, False, False, "bf16")
    y, resid, w_post, w_pre, gate = _inputs(case)
    for kw in (dict(w_post=w_post), dict(w_pre=w_pre), dict(gate=gate, rows_per_gate=5, w_pre=w_pre),
               dict(w_post=w_post, w_pre=w_pre, gate=gate, rows_per_gate=5)):
        for r in (resid, None):
            say(sorted(kw), r is not None)
            h, z = tb.tb_block_norm(y, r, alpha=-1.5, **kw)
            rh, rz = _ref(y, r, kw.get("w_post"), kw.get("w_pre"), kw.get("gate"), 5, -1.5, 1e-6, False, False)
            _check(h, rh, 20.0, False, "h")
            assert (z is None) == ("w_pre" not in kw)
            if z is not None:
                _check(z, rz, 80.0, False, "z")
    # the norm alone, of the residual stream; and without h
    h, z = tb.tb_block_norm(None, resid, w_pre=w_pre)
    assert h is None
    _check(z, _ref(None, resid, None, w_pre, None, 1, 1.0, 1e-6, False, False)[1], 40.0, False, "norm alone")
    h2, z2 = tb.tb_block_norm(y, resid, w_pre=w_pre, with_h=False)
    h3, z3 = tb.tb_block_norm(y, resid, w_pre=w_pre)
    assert h2 is None and torch.equal(z2, z3)
    # in place
    r = resid.clone()
    h4, _ = tb.tb_block_norm(y, r, w_pre=w_pre, h=r)
    torch.cuda.synchronize()
    assert h4.data_ptr() == r.data_ptr() and torch.equal(r, h3)


def test_block_norm_act8_is_the_bf16_result():
    rows, c = 3, 5120
    y, resid, w_post, w_pre, _ = _inputs((rows, c, 4, "f32", "f32", "bf16", None, True, True, "bf16"))
    kw = dict(w_post=w_post, w_pre=w_pre, y_parts=4, rotate_in=True, rotate_out=True)
    _, z = tb.tb_block_norm(y, resid, **kw)
    h, act = tb.tb_block_norm(y, resid, z_dtype=torch.uint8, **kw)
    torch.cuda.synchronize()
    bits = z.cpu().view(torch.int16).numpy().view(np.uint16)
    kept = oracle.numerics.bf16_bits_to_f64(act8_kept(bits))
    assert np.array_equal(act8_decode(act.cpu().numpy(), rows, c), kept)
    # and the bytes are those of encoding it afterwards
    assert torch.equal(act, tb.tb_act8_prep(z))


def test_block_norm_rows_of_zeros_and_of_nan():
    y = torch.zeros(3, 256, dtype=torch.bfloat16, device=DEV)
    resid = torch.zeros(3, 256, dtype=torch.bfloat16, device=DEV)
    y[1] = float("nan")
    y[2, 0] = float("inf")
    w = torch.ones(256, dtype=torch.bfloat16, device=DEV)
    h, z = tb.tb_block_norm(y, resid, w_post=w, w_pre=w)
    torch.cuda.synchronize()
    assert torch.all(h[0] == 0) and torch.all(z[0] == 0)      # eps keeps a row of zeros at 0
    assert torch.isnan(z[1]).all() and torch.isnan(h[1]).all()
    assert torch.isnan(h[2, 0])                              # inf / inf
    assert torch.isfinite(z[0]).all()


def test_block_norm_empty_and_out_given():
    w = torch.ones(128, dtype=torch.float32, device=DEV)
    e = torch.empty(0, 128, dtype=torch.float32, device=DEV)
    h, z = tb.tb_block_norm(e, e, w_pre=w)
    assert h.shape == (0, 128) and z.shape == (0, 128)
    y = torch.randn(2, 128, device=DEV)
    hh, zz = torch.empty(2, 128, device=DEV), torch.empty(2, 128, dtype=torch.bfloat16, device=DEV)
    h, z = tb.tb_block_norm(y, y.clone(), w_pre=w, h=hh, z=zz)
    assert h is hh and z is zz
    with pytest.raises(tb.TBError):
        tb.tb_block_norm(y, y, w_pre=w, z=y)             # z over its input
    with pytest.raises(ValueError):
        tb.tb_block_norm(y, y, w_pre=w[:64])
    with pytest.raises(ValueError):
        tb.tb_block_norm(y.t(), None, w_pre=w)
    with pytest.raises(TypeError):
        tb.tb_block_norm(y.double(), None, w_pre=w)


def test_block_norm_on_a_stream_and_in_a_graph():
    y, resid, w_post, w_pre, _ = _inputs((9, 1024, 2, "f32", "bf16", "bf16", None, True, True, "bf16"))
    kw = dict(w_post=w_post, w_pre=w_pre, y_parts=2, rotate_in=True, rotate_out=True)
    ref = tb.tb_block_norm(y, resid, **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = tb.tb_block_norm(y, resid, stream=s, **kw)
    s.synchronize()
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    h, z = torch.empty_like(ref[0]), torch.empty_like(ref[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        tb.tb_block_norm(y, resid, h=h, z=z, **kw)
    for _ in range(3):
        h.zero_()
        z.zero_()
        y.normal_()
        g.replay()
        torch.cuda.synchronize()
        e = tb.tb_block_norm(y, resid, **kw)
        assert torch.equal(h, e[0]) and torch.equal(z, e[1])

"""GPU parity of the 4-bit cache: its codes bit for bit, what is read back, and
the attention over it.

Codes, scales and offsets are those of the 64-bit formula: bf16 inputs are exact
in it, and numpy's division and rounding to float16 are correct ones.

Bounds of the attention as for the 8-bit cache (weights as fp16, 2^-11), e =
2^-24; a query element below 2^-24 of its row's largest is off by at most half
of 2^-34 of it, times the largest key channel, for each of d channels.  fp16
weights below 2^-14 are multiples of 2^-24, off by half of that; a row's largest
is at least 2^11 (chunks: relative to a maximum 11 binades above 1, which may lag
behind by less than 4 more; few rows: 2^15).  So a weight is off by at most
2^-36 of the largest, which the sum of the weights is not below, and an output by
2^-36 of the sum of the magnitudes of the values, however small their weights.
"""

import numpy as np
import pytest
import torch

import oracle
from gpu_util import DEV, host_f64, say
from test_gpu_paged import SHAPES, Case
from ternary_weights_hadamard_amd import tb

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
S = oracle.serving


def device(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


class Case4(Case):
    """The pool of a bf16 case in 4 bits; what no sequence holds has NaN scales."""

    def __init__(self, lens, hq, hkv, d, page, seed=0, spread=1.0, **kw):
        super().__init__(lens, hq, hkv, d, page, "bf16", seed=seed, **kw)
        k, v = host_f64(self.k) * spread, host_f64(self.v).transpose(0, 1, 3, 2) * spread
        self.hold(k, v)

    def hold(self, k, v):
        """Keys and values [pages, heads, page, d] as the pool."""
        kc, ks, ko = S.codes4(k)
        vc, vs, vo = S.codes4(v)
        self.k, self.k_scale = device(kc), device(np.stack([ks, ko], -1))
        self.v, self.v_scale = device(vc.transpose(0, 1, 3, 2)), device(np.stack([vs, vo], 2))

    def values(self):
        """What the pool stands for: keys [pages, heads, page, d], values [pages, heads, d, page]."""
        ks, vs = self.k_scale.cpu().numpy(), self.v_scale.cpu().numpy()
        k = S.values4(self.k.cpu().numpy(), ks[..., 0], ks[..., 1])
        v = S.values4(self.v.cpu().numpy().transpose(0, 1, 3, 2), vs[:, :, 0], vs[:, :, 1])
        return k, v.transpose(0, 1, 3, 2)

    def check(self, out, lse, scale=None, window=0, what=""):
        torch.cuda.synchronize()
        k, v = self.values()
        q = host_f64(self.q.contiguous())
        scale = self.d ** -0.5 if scale is None else scale
        ref, rl, mean, size = S.paged_attention(q, k, v, self.table, self.cu, self.kv, scale, window)
        low = self.d * 2.0 ** -35 * np.abs(q).max(-1) * np.nanmax(np.abs(k), initial=0.0) * abs(scale)
        weight = 2 * ((self.d + 4) * E * size + low)[..., None] + 2.0 ** -11 + (self.max_kv + 64) * E
        half = np.abs(ref) * 2.0 ** -8 if out.dtype == torch.bfloat16 else 0.0
        small = 2.0 ** -36 * self.max_kv * np.nanmax(np.abs(v), initial=0.0)
        bound = weight * mean + half + small + 1e-30
        got, gl = host_f64(out), host_f64(lse)
        err = np.abs(got - ref)
        say(f"  {what}: max err {err.max(initial=0):.3e}, of the bound {np.max(err / bound, initial=0):.2f}")
        assert np.all(np.isfinite(got)), what
        assert np.all(err <= bound), what
        empty = np.isneginf(rl)
        assert np.array_equal(np.isneginf(gl), empty), what
        assert np.all(got[empty] == 0.0), what
        lb = (self.d + 4) * E * size + low + (self.max_kv + 64) * E + 4 * E * np.abs(np.where(empty, 0, rl))
        assert np.all(np.abs(gl[~empty] - rl[~empty]) <= lb[~empty]), what


APPENDS = [
    # lens, heads, d, page
    ([(1, 1)], 1, 128, 16),
    ([(1, 700), (1, 33), (0, 5), (1, 1)], 8, 128, 64),
    ([(3, 3), (5, 100), (16, 31), (2, 64)], 2, 64, 32),
    ([(33, 33), (7, 129), (64, 200)], 5, 128, 16),
    ([(130, 333), (1, 70), (257, 257)], 3, 64, 128),
    ([(5, 2), (30, 20), (2, 1)], 4, 128, 16),                # tokens before position 0 have no place
    ([(77, 1100)], 9, 128, 1024),
]


def holds(pages, table, page, kv):
    """Which [page, slot] belong to positions kv of each sequence."""
    m = np.zeros((pages, page), bool)
    for b, xs in enumerate(kv):
        for x in xs:
            m[table[b, x // page], x % page] = True
    return m


@pytest.mark.parametrize("case", APPENDS, ids=lambda c: f"{len(c[0])}x{max(n for n, _ in c[0])}-h{c[1]}-d{c[2]}-p{c[3]}")
def test_append_codes(case):
    lens, heads, d, page = case
    say(f"append4 {case}")
    c = Case4(lens, heads, heads, d, page, seed=3)
    # rows with what rounds hardest: equal channels, an infinity, a NaN, halves of a step, far values
    k, v = c.new_k.clone(), c.new_v.clone()
    for t, x in ((k, 0), (v, 1)):
        n = t.shape[0]
        t[x % n, 0] = 2.5
        t[(x + 2) % n, 0, :3] = torch.tensor([float("inf"), -1.0, 100.0])
        t[(x + 4) % n, -1, 7] = float("nan")
        t[(x + 5) % n, -1] = torch.arange(d, device=DEV).to(torch.bfloat16) % 31 / 2     # scale 1, all ties
        t[(x + 6) % n, 0] *= 1e30
        t[(x + 7) % n, 0] *= 1e-30
    before = [t.cpu().numpy().copy() for t in (c.k, c.v, c.k_scale, c.v_scale)]
    tb.tb_paged_append(k, v, c.k, c.v, c.table_d, c.cu_d, c.kv_d, c.max_q, k_scale=c.k_scale, v_scale=c.v_scale)
    torch.cuda.synchronize()
    kc, ks, ko = S.codes4(host_f64(k))
    vc, vs, vo = S.codes4(host_f64(v))
    want = before
    for b, (n, kv) in enumerate(lens):
        for r, pos in S.paged_rows(c.cu, c.kv, b):
            at = S.paged_slot(c.table, page, c.pages, b, pos)
            if at is None:
                continue
            p, s = at
            want[0][p, :, s], want[1][p, :, :, s] = kc[r], vc[r]
            want[2][p, :, s, 0], want[2][p, :, s, 1] = ks[r], ko[r]
            want[3][p, :, 0, s], want[3][p, :, 1, s] = vs[r], vo[r]
    for got, w, what in zip((c.k, c.v, c.k_scale, c.v_scale), want, ("k", "v", "k_scale", "v_scale")):
        got = got.cpu().numpy()
        if got.dtype == np.float16:  # any NaN is one
            same = (got.view(np.uint16) == w.view(np.uint16)) | (np.isnan(got) & np.isnan(w))
        else:
            same = got == w
        assert same.all(), f"{what}: {int((~same).sum())} of {same.size} differ"


@pytest.mark.parametrize("cache", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("case", APPENDS[1:], ids=lambda c: f"{len(c[0])}x{max(n for n, _ in c[0])}-h{c[1]}-d{c[2]}-p{c[3]}")
def test_read(case, dtype, cache):
    lens, heads, d, page = case
    say(f"read {case} {dtype} {cache}")
    c = Case4(lens, heads, heads, d, page) if cache == "int4" else Case(lens, heads, heads, d, page, cache)
    if cache == "int4":
        kr, vr = c.values()
    else:
        kr, vr = host_f64(c.k.float()), host_f64(c.v.float())
        if cache == "fp8":
            kr = (kr.astype(np.float32) * c.k_scale.cpu().numpy()[None, :, None, None]).astype(np.float64)
            vr = (vr.astype(np.float32) * c.v_scale.cpu().numpy()[None, :, None, None]).astype(np.float64)
    counts = [kv if b % 2 == 0 else n for b, (n, kv) in enumerate(lens)]    # whole sequences, and new tokens
    cu = np.concatenate([[0], np.cumsum(counts)])
    total = int(cu[-1]) + 2
    k = torch.full((total, heads, d), 7.0, dtype=dtype, device=DEV)
    v = torch.full_like(k, 9.0)
    cu_d = device(cu.astype(np.int32))
    got = tb.tb_paged_read(c.k, c.v, c.table_d, cu_d, c.kv_d, total, max(counts), c.k_scale, c.v_scale, k, v)
    assert got[0] is k and got[1] is v
    wk, wv = np.full((total, heads, d), 7.0), np.full((total, heads, d), 9.0)
    for b in range(len(lens)):
        for r, pos in S.paged_rows(cu, c.kv, b):
            at = S.paged_slot(c.table, page, c.pages, b, pos)
            if at is not None:
                wk[r], wv[r] = kr[at[0], :, at[1]], vr[at[0], :, :, at[1]]
    wk, wv = (torch.from_numpy(w).float().to(dtype).double().numpy() for w in (wk, wv))
    for got, w, other in ((k, wk, 0), (v, wv, 1)):
        assert np.array_equal(host_f64(got), w)
    # one of the two alone
    only = torch.zeros_like(k)
    args = tb._paged_cache("test", c.k, c.k, c.v, c.table_d, cu_d, c.kv_d, max(counts), c.k_scale, c.v_scale)
    args.total_q = total
    assert tb.lib().tb_paged_read(args, None, only.data_ptr(), tb.TB_F32 if dtype == torch.float32 else tb.TB_BF16,
                                  torch.cuda.current_stream().cuda_stream) == 0
    torch.cuda.synchronize()
    held = np.array([any(cu[b] <= r < cu[b + 1] and c.kv[b] - (cu[b + 1] - r) >= 0 for b in range(len(lens))) for r in range(total)])
    assert np.array_equal(host_f64(only)[held], wv[held]) and not host_f64(only)[~held].any()


@pytest.mark.parametrize("split", [True, False])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{len(s[0])}x{max(n for n, _ in s[0])}-{max(k for _, k in s[0])}-"
                                                         f"h{s[1]}.{s[2]}-d{s[3]}-p{s[4]}-w{s[5]}")
def test_attention_matches_oracle(shape, split):
    lens, hq, hkv, d, page, window = shape
    say(f"attention4 {shape} {split}")
    c = Case4(lens, hq, hkv, d, page)
    kw = {} if split else dict(workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    for dtype in (torch.float32, torch.bfloat16):
        out, lse = c.attend(window=window, out_dtype=dtype, **kw)
        c.check(out, lse, window=window, what=str(dtype))


@pytest.mark.parametrize("lens", [[(1, 300), (2, 70)], [(40, 300), (1, 70), (200, 260)]])
@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0, 1e-30])
def test_attention_scales(lens, scale):
    say(f"attention4 scale {scale} {lens}")
    c = Case4(lens, 8, 2, 128, 16, seed=2)
    out, lse = c.attend(scale=scale, out_dtype=torch.float32)
    c.check(out, lse, scale=scale, what=f"scale {scale}")


@pytest.mark.parametrize("lens", [[(1, 300), (2, 70)], [(40, 300), (200, 260)]])
@pytest.mark.parametrize("size", [1e-38, 1e-20, 1e-3, 1e5, 1e25])
def test_queries_of_any_size(lens, size):
    """fp16 queries are in units of their row: neither large nor small ones are lost."""
    say(f"attention4 queries of {size} {lens}")
    c = Case4(lens, 4, 2, 64, 32, seed=5)
    mixed = torch.ones(c.total, 4, 1, device=DEV)
    mixed[::2, 1] = 1e3                                     # rows of one tile differ
    c.q = (c.q.float() * size * mixed).to(torch.bfloat16)
    scale = 0.3 / size if size > 1e-30 else 1.0             # 0.3 / 1e-38 is past fp32
    out, lse = c.attend(scale=scale, out_dtype=torch.float32)
    c.check(out, lse, scale=float(np.float32(scale)), what=f"size {size}")


@pytest.mark.parametrize("lens", [[(1, 300), (2, 70)], [(40, 300), (200, 260)]])
@pytest.mark.parametrize("spread", [1e-7, 1e-3, 300.0, 4000.0])
def test_values_of_any_size(lens, spread):
    """Scales among fp16's subnormal numbers, and large ones."""
    say(f"attention4 values of {spread} {lens}")
    c = Case4(lens, 4, 2, 128, 16, seed=6, spread=spread)
    out, lse = c.attend(scale=0.1 / max(spread, 1e-3), out_dtype=torch.float32)
    c.check(out, lse, scale=float(np.float32(0.1 / max(spread, 1e-3))), what=f"spread {spread}")


@pytest.mark.parametrize("lens", [[(3, 300)], [(70, 300)]])
def test_nan_reaches_only_who_sees_it(lens):
    say(f"attention4 NaN {lens}")
    n, kv = lens[0]
    for which in ("k_scale", "v_scale"):
        c = Case4(lens, 4, 2, 64, 16, seed=1)
        want, _ = c.attend(out_dtype=torch.float32)
        pos = kv - 2                                        # the last two tokens see it
        at = (c.table[0, pos // 16], pos % 16)
        t = getattr(c, which)
        if which == "k_scale":
            t[at[0], 1, at[1]] = float("nan")
        else:
            t[at[0], 1, :, at[1]] = float("nan")
        got, _ = c.attend(out_dtype=torch.float32)
        bad = torch.isnan(got)
        assert bad[-2:, 2:].all() and not bad[-2:, :2].any() and not bad[:-2].any()
        assert torch.equal(got[:-2], want[:-2]) and torch.equal(got[-2:, :2], want[-2:, :2])


def test_infinite_values_that_nobody_sees():
    """Scales that make infinities, where a position is not seen, or is past the end."""
    say("attention4 unseen infinities")
    for lens in ([(3, 300)], [(70, 300)]):
        c = Case4(lens, 4, 2, 64, 16, seed=1, poison=False)
        want, wl = c.attend(out_dtype=torch.float32, window=64)
        n, kv = lens[0]
        for pos in [0, 17, kv - n - 64]:
            c.v_scale[c.table[0, pos // 16], :, 0, pos % 16] = 60000.0
            c.k_scale[c.table[0, pos // 16], :, pos % 16, 0] = -60000.0
        last = (kv - 1) // 16
        for slot in range(kv % 16, 16):
            c.v_scale[c.table[0, last], :, :, slot] = float("inf")
            c.k_scale[c.table[0, last], :, slot] = float("-inf")
        got, gl = c.attend(out_dtype=torch.float32, window=64)
        assert torch.equal(got, want) and torch.equal(gl, wl)


def test_wrong_tables_stay_inside():
    """Entries of the table, lengths and offsets that lead nowhere: nothing outside is read or written."""
    say("wrong tables")
    c = Case4([(2, 100), (40, 90), (1, 64)], 4, 2, 64, 16, seed=4)
    c.table[0, 3], c.table[1, 2], c.table[2, 0] = 10 ** 6, -5, 2 ** 31 - 1
    c.kv[2] = 10 ** 6
    c.ints()
    before = [t.clone() for t in (c.k, c.v, c.k_scale, c.v_scale)]
    out, lse = c.attend(out_dtype=torch.float32)
    kv = c.kv[2]
    c.kv[2] = min(kv, c.table.shape[1] * 16)                # positions past the table do not exist
    k, v = c.values()
    assert torch.isfinite(out[:42]).all()
    ref, _, _, _ = S.paged_attention(host_f64(c.q.contiguous())[:42], k, v, c.table[:2], c.cu[:3], c.kv[:2], 0.125, 0)
    assert np.abs(host_f64(out)[:42] - ref).max() < 2e-2
    c.append()
    torch.cuda.synchronize()
    changed = (c.k_scale != before[2]).any(dim=3).any(dim=1).cpu().numpy() & ~torch.isnan(before[2]).any(dim=3).any(dim=1).cpu().numpy()
    mine = holds(c.pages, c.table, 16, [range(98, 100), [x for x in range(50, 90) if x // 16 != 2], []])
    assert not (changed & ~mine).any()


def test_two_streams_and_graphs():
    """The same call on another stream, and captured and replayed, gives the same bits."""
    say("attention4 streams and graphs")
    for lens in ([(1, 2000)] * 5, [(200, 900), (3, 500)]):
        c = Case4(lens, 8, 2, 128, 16, seed=7)
        want, wl = c.attend()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        out, lse = c.attend(stream=side)
        side.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, wl)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            go, gl = c.attend()
        for _ in range(3):
            go.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(go, want) and torch.equal(gl, wl)

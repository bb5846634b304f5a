"""GPU parity of the rotary append.

Queries, e = 2^-24, in fp32 from exact bf16: the transform is seven additions of
numbers that are at most the sum of the head's magnitudes (7 e of that sum over
sqrt(128)) and a multiplication (e); cosine and sine are rounded once (e), the
factor's product with them and the two products of the rotation add 3 e: of at
most `size`, the sum of the magnitudes that go into an element.  Twice for
turn_out.  20 e of a head's largest possible element, and half a bf16 step (2^-8).
Keys of a bf16 cache have the same bound.  Codes of the other caches are of the
64-bit formula: an element whose quotient is no nearer than 1e-9 to the middle
between two codes has the oracle's; scales the same.
"""

import numpy as np
import pytest
import torch

import oracle
from gpu_util import DEV, host_f64, say
from test_gpu_cache4 import Case4, device, holds
from test_gpu_paged import Case
from ternary_weights_hadamard_amd import tb

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
S = oracle.serving


def turned(x):
    return oracle.hadamard.fwht_dense(x.reshape(-1, 128)).reshape(x.shape)


class Rotary:
    def __init__(self, lens, hq, hkv, d, page, cache, rot, neighbours=False, turn=(False, False, False), factor=1.0,
                 base=10000.0, seed=0):
        self.c = c = (Case4(lens, hq, hkv, d, page, seed=seed) if cache == "int4" else
                      Case(lens, hq, hkv, d, page, cache, seed=seed))
        self.cache, self.rot, self.neighbours, self.turn, self.factor = cache, rot, neighbours, turn, factor
        self.freq = tb.tb_rotary_frequencies(rot, base)[0].to(DEV) if rot else None
        self.before = [t.clone() for t in (c.k, c.v)] + ([c.k_scale.clone(), c.v_scale.clone()] if cache == "int4" else [])

    def run(self, **kw):
        c, t = self.c, self.turn
        a = dict(factor=self.factor, neighbours=self.neighbours, turn_in=t[0], turn_out=t[1], turn_v=t[2], k_scale=c.k_scale,
                 v_scale=c.v_scale)
        a.update(kw)
        return tb.tb_paged_append_rotary(c.q, c.new_k, c.new_v, c.k, c.v, c.table_d, c.cu_d, c.kv_d, c.max_q, self.freq, **a)

    def reference(self):
        """Queries, keys and values in 64 bits, and the largest that an element may be."""
        c, t = self.c, self.turn
        pos = np.zeros(c.total, np.int64)
        for b in range(len(c.lens)):
            for r, x in S.paged_rows(c.cu, c.kv, b):
                pos[r] = x
        f = host_f64(self.freq) if self.rot else np.zeros(0)
        factor = float(np.float32(self.factor))
        out = []
        for x in (c.q, c.new_k):
            x = host_f64(x.contiguous())
            size = np.abs(x).sum(-1, keepdims=True) / (128 ** 0.5 if t[0] else 1)
            if t[0]:
                x = turned(x)
            x = S.rotary(x, pos, f, factor, self.neighbours)
            size = size * max(1.0, 2 * factor) * (128 ** 0.5 if t[1] else 1)
            if t[1]:
                x = turned(x)
            out += [x, size]
        v = host_f64(c.new_v.contiguous())
        return out + [turned(v) if t[2] else v]

    def check(self, q):
        torch.cuda.synchronize()
        c, page = self.c, self.c.page
        rq, qs, rk, ks, rv = self.reference()
        err = np.abs(host_f64(q) - rq)
        bound = 20 * E * qs + 2.0 ** -8 * np.abs(rq)
        say(f"  queries: max err {err.max(initial=0):.2e}, of the bound {np.max(err / bound, initial=0):.2f}")
        assert np.all(err <= bound)
        at = [(r, S.paged_slot(c.table, page, c.pages, b, x)) for b in range(len(c.lens)) for r, x in S.paged_rows(c.cu, c.kv, b)]
        at = [(r, p, s) for r, w in at if w is not None for p, s in [w]]
        rows, pages, slots = (np.array([x[i] for x in at], np.int64) for i in range(3))
        mine = np.zeros((c.pages, page), bool)
        mine[pages, slots] = True
        for name, ref, now, before in (("k", rk, c.k, self.before[0]), ("v", rv, c.v, self.before[1])):
            bits = lambda t: t.view(torch.uint8 if t.element_size() == 1 else torch.int16).cpu().numpy()  # noqa: E731
            order = lambda a: a if name == "k" else a.transpose(0, 1, 3, 2)  # noqa: E731  [pages, heads, page, d]
            got, old = order(bits(now)), order(bits(before))
            keep = ~mine[:, None, :, None]
            assert np.array_equal(np.where(keep, got, 0), np.where(keep, old, 0)), f"{name}: other positions changed"
            got, want = got[pages, :, slots], ref[rows]
            if self.cache == "bf16":
                value = oracle.numerics.bf16_bits_to_f64(got.view(np.uint16))
                assert np.all(np.abs(value - want) <= 2.0 ** -8 * np.abs(want) + (20 * E * ks[rows] if name == "k" or self.turn[2] else 0))
            elif self.cache == "fp8":
                s = (c.k_scale if name == "k" else c.v_scale).double().cpu().numpy()[None, :, None]
                x = np.clip(want / s, -448, 448)
                codes = lambda a: torch.from_numpy(a).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()  # noqa: E731
                low, high = codes(x * (1 - 1e-9)), codes(x * (1 + 1e-9))
                assert np.all((got == low) | (got == high)), f"{name}: {np.sum((got != low) & (got != high))} codes"
            else:
                scale = (c.k_scale if name == "k" else c.v_scale).cpu().numpy()
                old = self.before[2 if name == "k" else 3].cpu().numpy()
                pick = lambda a: (a if name == "k" else a.transpose(0, 1, 3, 2))  # noqa: E731
                scale, old = pick(scale), pick(old)
                keep = ~mine[:, None, :, None] & ~np.isnan(old)
                assert np.array_equal(np.where(keep, scale, 0), np.where(keep, old, 0)), f"{name}: other scales changed"
                codes, ws, wo = S.codes4(want)
                scale = scale[pages, :, slots]
                assert np.array_equal(scale[..., 0], ws) and np.array_equal(scale[..., 1], wo), f"{name}: scales"
                diff = got != codes
                if diff.any():
                    n = (want - wo.astype(np.float64)[..., None]) / ws.astype(np.float64)[..., None]
                    near = np.abs(n - np.floor(n) - 0.5) < 1e-9
                    d8 = near.reshape(near.shape[:-1] + (-1, 2, 4)).any(-2).reshape(diff.shape)
                    assert not (diff & ~d8).any(), f"{name}: {int(diff.sum())} codes"


CASES = [
    # lens, heads_q, heads_kv, d, page, rotary_dim, neighbours, turns, factor
    ([(1, 1)], 1, 1, 128, 16, 128, False, (0, 0, 0), 1.0),
    ([(1, 700), (1, 33), (0, 5), (1, 1)], 40, 8, 128, 64, 128, False, (1, 1, 1), 1.0),
    ([(3, 3), (5, 100), (16, 31), (2, 64)], 4, 2, 64, 32, 64, True, (0, 0, 0), 1.25),
    ([(9, 5000), (1, 70)], 6, 2, 64, 16, 48, False, (0, 0, 0), 1.0),
    ([(33, 33), (7, 129), (64, 200)], 10, 5, 128, 16, 96, True, (1, 0, 0), 0.5),
    ([(130, 333), (1, 70), (257, 257)], 3, 3, 64, 128, 16, False, (0, 0, 0), 1.0),
    ([(5, 2), (30, 20), (2, 1)], 8, 4, 128, 16, 128, False, (0, 1, 1), 1.0),   # tokens before position 0 have no place
    ([(77, 1100), (17, 77)], 9, 9, 128, 1024, 32, False, (1, 1, 0), 1.0),
    ([(20, 60)], 41, 1, 128, 64, 0, False, (1, 0, 1), 1.0),                    # no positions: the basis alone
    ([(70, 70000)], 5, 1, 128, 64, 128, True, (0, 0, 0), 1.1),                 # far positions
]


@pytest.mark.parametrize("cache", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}x{max(n for n, _ in c[0])}-h{c[1]}.{c[2]}-d{c[3]}-p{c[4]}"
                                                      f"-r{c[5]}{'n' if c[6] else ''}-t{''.join(str(t) for t in c[7])}")
def test_matches_oracle(case, cache):
    lens, hq, hkv, d, page, rot, neighbours, turn, factor = case
    say(f"rotary {case} {cache}")
    r = Rotary(lens, hq, hkv, d, page, cache, rot, neighbours, tuple(bool(t) for t in turn), factor)
    r.check(r.run())


@pytest.mark.parametrize("cache", ["bf16", "int4"])
def test_far_positions(cache):
    """Angles of positions up to 2^30 - 1 and frequencies above 1 are reduced in 64 bits."""
    say(f"rotary far {cache}")
    # a table of one page a sequence cannot reach them: keys have no place, queries are rotated
    r = Rotary([(3, 30), (20, 40)], 2, 1, 64, 16, cache, 64)
    c = r.c
    r.freq *= 3.7
    c.kv = [2 ** 30 - 1, 2 ** 27 + 11]
    c.ints()
    r.check(r.run())


@pytest.mark.parametrize("lens", [[(70, 70), (200, 300)], [(16, 90), (9, 70), (3, 3), (16, 16), (16, 40)]])
def test_codes_far_from_zero(lens):
    """One channel far above the others becomes, turned, the same large number in
    every channel with a little on it: up to thousands of steps from 0."""
    say(f"far from zero {lens}")
    r = Rotary(lens, 2, 8, 128, 64, "int4", 0, turn=(False, True, True), seed=11)
    for t in (r.c.new_k, r.c.new_v):
        t.mul_(0.25)
        n = t.shape[0] * t.shape[1]
        t[..., 0] = torch.linspace(100.0, 45000.0, n, device=DEV).view(t.shape[:2]).to(torch.bfloat16)
        t[::2, :, 0].neg_()
    r.check(r.run())


@pytest.mark.parametrize("turn", [(True, True, True), (False, False, False)])
def test_codes_of_many_rows(turn):
    """Enough rows that some scales and offsets lie next to where fp16 rounds."""
    say(f"many rows {turn}")
    r = Rotary([(600, 700), (500, 500)], 2, 16, 128, 64, "int4", 128, turn=turn, seed=12)
    r.check(r.run())


def test_without_queries_and_in_place():
    say("rotary without queries")
    for lens in ([(3, 30)], [(40, 60)]):
        a = Rotary(lens, 4, 2, 128, 16, "int4", 128, turn=(True, True, True))
        b = Rotary(lens, 4, 2, 128, 16, "int4", 128, turn=(True, True, True))
        a.run()
        c = b.c
        assert tb.tb_paged_append_rotary(None, c.new_k, c.new_v, c.k, c.v, c.table_d, c.cu_d, c.kv_d, c.max_q, b.freq,
                                         turn_in=True, turn_out=True, turn_v=True, k_scale=c.k_scale, v_scale=c.v_scale) is None
        for x, y in ((a.c.k, c.k), (a.c.v, c.v), (a.c.k_scale.view(torch.int16), c.k_scale.view(torch.int16)),
                     (a.c.v_scale.view(torch.int16), c.v_scale.view(torch.int16))):
            assert torch.equal(x, y)


def test_rows_of_no_sequence_stay():
    """Tokens behind the last sequence and past max_q: their queries are left, their keys not written."""
    say("rotary other rows")
    for most in (4, 40):
        r = Rotary([(most, 100), (most, 90)], 4, 2, 64, 16, "bf16", 64)
        c = r.c
        c.cu_d[2] -= 2                                      # two rows of no sequence
        out = torch.full_like(c.q, 7.0).contiguous()
        c.max_q = most - 1
        r.run(q_out=out)
        torch.cuda.synchronize()
        assert (out[most - 1] == 7.0).all() and (out[-2:] == 7.0).all()
        assert (out[:most - 1] != 7.0).any(dim=-1).all() and (out[most:-2] != 7.0).any(dim=-1).all()
        changed = (c.k.view(torch.int16) != r.before[0].view(torch.int16)).any(dim=3).any(dim=1).cpu().numpy()
        mine = holds(c.pages, c.table, 16, [range(100 - most, 99), range(92 - most, 90)])
        assert not (changed & ~mine).any()


def test_wrong_tables_stay_inside():
    say("rotary wrong tables")
    for cache in ("bf16", "fp8", "int4"):
        for lens in ([(2, 100), (16, 90)], [(40, 100), (30, 90)]):
            r = Rotary(lens, 4, 2, 64, 16, cache, 64)
            c = r.c
            c.table[0, 6], c.table[1, 5] = 10 ** 6, -1
            c.ints()
            c.cu_d[1] += 10 ** 6
            r.run()
            torch.cuda.synchronize()
            c.ints()
            want = r.reference()[0]
            r2 = r.run()
            torch.cuda.synchronize()
            assert np.abs(host_f64(r2) - want).max() < 0.05


def test_streams_and_graphs():
    say("rotary streams and graphs")
    for lens in ([(1, 40), (3, 60)], [(50, 80), (3, 60)]):
        a, b = (Rotary(lens, 8, 2, 128, 16, "int4", 128, turn=(True, True, True)) for _ in range(2))
        want = a.run()
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        got = b.run(stream=side)
        side.synchronize()
        assert torch.equal(got, want) and torch.equal(a.c.k, b.c.k) and torch.equal(a.c.v, b.c.v)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = b.run()
        for k in range(3):
            b.c.q.mul_(-1)
            out.zero_()
            b.c.k.zero_(), b.c.v.zero_()
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, -want if k % 2 == 0 else want)
            mine = holds(b.c.pages, b.c.table, 16, [range(kv - n, kv) for n, kv in lens])
            m = device(mine)[:, None, :, None]
            assert torch.equal(b.c.k, torch.where(m, a.c.k, torch.zeros_like(a.c.k)))


@pytest.mark.parametrize("cache", ["bf16", "fp8", "int4"])
def test_cache_then_attention(cache):
    """A prompt in chunks and tokens one by one, rotated into the cache and attended
    to, against all of it at once in 64 bits.  The attention is bounded by its own
    test; here bf16 queries, keys and values (2^-8 of each, sums of 128 products at
    scores of about 1) and the cache's steps: 4 bits change outputs by a share of
    the values' size that is not derived, so that the comparison is with the
    cache's own values."""
    say(f"rotary and attention {cache}")
    hq, hkv, d, page, total = 4, 2, 128, 16, 150
    g = torch.Generator().manual_seed(3)
    fused = torch.randn((total, hq + 2 * hkv, d), generator=g).to(torch.bfloat16).to(DEV)
    pages = 2 * (total // page + 2)
    kind = {"bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn, "int4": torch.uint8}[cache]
    width = d // 2 if cache == "int4" else d
    k = torch.zeros((pages, hkv, page, width), dtype=torch.uint8 if cache != "bf16" else kind, device=DEV).view(kind)
    v = torch.zeros((pages, hkv, width, page), dtype=torch.uint8 if cache != "bf16" else kind, device=DEV).view(kind)
    ks = vs = None
    if cache == "fp8":
        ks = vs = torch.full((hkv,), 1 / 32, device=DEV)
    if cache == "int4":
        ks, vs = (torch.zeros(s, dtype=torch.float16, device=DEV) for s in ((pages, hkv, page, 2), (pages, hkv, 2, page)))
    table = torch.randperm(pages, generator=g)[:pages // 2][None].to(torch.int32).to(DEV)
    freq = tb.tb_rotary_frequencies(d)[0].to(DEV)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    outs, qs, at = [], [], 0
    for n in [70, 33, 1, 1, 5, 1, 39]:
        q, kk, vv = fused[at:at + n].split([hq, hkv, hkv], dim=1)
        at += n
        where = (k, v, table, ints([0, n]), ints([at]))
        q = tb.tb_paged_append_rotary(q, kk, vv, *where, n, freq, turn_in=True, turn_out=True, turn_v=True, k_scale=ks, v_scale=vs)
        outs.append(tb.tb_paged_attention(q, *where, n, at, k_scale=ks, v_scale=vs, out_dtype=torch.float32))
        qs.append(q)
    assert at == total
    kr, vr = (host_f64(t) for t in tb.tb_paged_read(k, v, table, ints([0, total]), ints([total]), total, total, ks, vs,
                                                    out_dtype=torch.float32))
    # what is held is what was meant, to the cache's step
    pos = np.arange(total)
    x = turned(host_f64(fused))
    want_k = turned(S.rotary(x[:, hq:hq + hkv], pos, host_f64(freq), 1.0, False))
    step = {"bf16": 2.0 ** -8, "fp8": 2.0 ** -4}.get(cache, 0) * np.abs(want_k) + {"fp8": 2.0 ** -15, "int4": 0.6 * np.ptp(want_k, -1, keepdims=True) / 15}.get(cache, 1e-5)
    assert np.all(np.abs(kr - want_k) <= step)
    q = host_f64(torch.cat(qs))
    for h in range(hq):
        s = q[:, h] @ kr[:, h // 2].T * d ** -0.5
        s[np.triu_indices(total, 1)] = -np.inf
        w = np.exp(s - s.max(1, keepdims=True))
        ref = w @ vr[:, h // 2] / w.sum(1, keepdims=True)
        mean = w @ np.abs(vr[:, h // 2]) / w.sum(1, keepdims=True)
        # weights to 2^-8 at most, fp32 sums of 128 products
        assert np.all(np.abs(host_f64(torch.cat(outs))[:, h] - ref) <= (2.0 ** -8 + 1e-4) * mean)


def test_refusals():
    r = Rotary([(2, 30)], 4, 2, 64, 16, "int4", 64)
    c = r.c
    args = (c.k, c.v, c.table_d, c.cu_d, c.kv_d, 2)
    good = dict(k_scale=c.k_scale, v_scale=c.v_scale)
    call = lambda q, k, v, freq, **kw: tb.tb_paged_append_rotary(q, k, v, *args, freq, **dict(good, **kw))  # noqa: E731
    with pytest.raises(ValueError):
        call(c.q, c.new_k, c.new_v[:1], r.freq)
    with pytest.raises(ValueError):
        call(c.q[:1], c.new_k, c.new_v, r.freq)
    with pytest.raises(ValueError):
        call(c.q, c.new_k, c.new_v, r.freq.double())
    with pytest.raises(ValueError):
        call(c.q, c.new_k, c.new_v, r.freq, k_scale=None)
    with pytest.raises(ValueError):
        call(c.q, c.new_k, c.new_v, r.freq, k_scale=c.k_scale.float())
    with pytest.raises(ValueError):
        call(None, c.new_k, c.new_v, r.freq, q_out=c.q.contiguous())
    with pytest.raises(tb.TBError):
        call(c.q, c.new_k, c.new_v, r.freq, turn_in=True)   # heads of 64
    with pytest.raises(tb.TBError):
        call(c.q, c.new_k, c.new_v, r.freq[:12])
    with pytest.raises(TypeError):
        tb.tb_paged_append(c.new_k, c.new_v, c.k.view(torch.int8), c.v.view(torch.int8), *args[2:], **good)

"""GPU parity of the paged cache and of the attention over it.

Appended codes are checked bit for bit (bf16 copies; e4m3 by torch's own
conversion of the fp32 quotient).

Bounds of the attention, e = 2^-24: a score is a sum of d exact products in
fp32, off by at most d e of the sum of their magnitudes (`size`, from the
oracle), scaled and subtracted with 4 e more; twice that (numerator and
denominator) is the relative error of a weight, plus the weight's rounding:
2^-11 as fp16 (an 8-bit cache) or 2^-8 as bf16, the most that any path uses;
sums over the positions add one e for each of their terms.  All of it times the
weighted mean magnitude of the values (`mean`).  A bf16 output adds half a
step, 2^-8.
"""

import numpy as np
import pytest
import torch

import oracle
from gpu_util import DEV, host_f64, say
from ternary_weights_hadamard_amd import tb

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
KIND = {"bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn, "f32": torch.float32}


class Case:
    """A pool of pages with sequences scattered over it.  `lens` are (new
    tokens, positions) of each; unused pages, table entries and the slots past
    a sequence's end hold what must not matter."""

    def __init__(self, lens, hq, hkv, d, page, cache, seed=0, poison=True, extra=3):
        rng = np.random.default_rng(seed + sum(kv for _, kv in lens) + hq + d)
        self.lens, self.hq, self.hkv, self.d, self.page = lens, hq, hkv, d, page
        self.n, self.kv = [n for n, _ in lens], [kv for _, kv in lens]
        need = [-(-kv // page) for kv in self.kv]
        self.pages = sum(need) + extra
        ids = rng.permutation(self.pages)
        width = max(need) + 2
        self.table = np.full((len(lens), width), -7, np.int64)
        at = 0
        for b, m in enumerate(need):
            self.table[b, :m] = ids[at:at + m]
            at += m
        self.cu = np.concatenate([[0], np.cumsum(self.n)])
        self.total, self.max_q, self.max_kv = int(self.cu[-1]), max(max(self.n), 1), max(max(self.kv), 1)
        kind = KIND[cache]
        shape = (self.pages, hkv, page, d)
        g = torch.Generator().manual_seed(seed)
        k = torch.randn(shape, generator=g)
        v = torch.randn((self.pages, hkv, d, page), generator=g)
        if poison:  # what no sequence holds is NaN
            held = torch.zeros(self.pages, page, dtype=torch.bool)
            for b, kv in enumerate(self.kv):
                for x in range(kv):
                    held[self.table[b, x // page], x % page] = True
            k[~held[:, None, :, None].expand(shape)] = float("nan")
            v[~held[:, None, None, :].expand(v.shape)] = float("nan")
        self.k_scale = self.v_scale = None
        if cache == "fp8":
            k, v = k * 16, v * 16
            self.k_scale = torch.from_numpy(rng.uniform(0.03, 0.1, hkv).astype(np.float32)).to(DEV)
            self.v_scale = torch.from_numpy(rng.uniform(0.03, 0.1, hkv).astype(np.float32)).to(DEV)
        self.k, self.v = k.to(kind).to(DEV), v.to(kind).to(DEV)
        fused = torch.randn((self.total, hq + 2 * hkv, d), generator=g).to(torch.bfloat16).to(DEV)
        self.q, self.new_k, self.new_v = fused[:, :hq], fused[:, hq:hq + hkv], fused[:, hq + hkv:]
        self.ints()

    def ints(self):
        i = lambda a: torch.from_numpy(np.asarray(a).astype(np.int32)).to(DEV)  # noqa: E731
        self.table_d, self.cu_d, self.kv_d = i(self.table), i(self.cu), i(self.kv)

    def attend(self, **kw):
        kw.setdefault("with_lse", True)
        return tb.tb_paged_attention(self.q, self.k, self.v, self.table_d, self.cu_d, self.kv_d, self.max_q, self.max_kv,
                                     k_scale=self.k_scale, v_scale=self.v_scale, **kw)

    def append(self, **kw):
        tb.tb_paged_append(self.new_k, self.new_v, self.k, self.v, self.table_d, self.cu_d, self.kv_d, self.max_q,
                           k_scale=self.k_scale, v_scale=self.v_scale, **kw)

    def reference(self, scale=None, window=0):
        k, v = self.k.float().double().cpu().numpy(), self.v.float().double().cpu().numpy()
        if self.k_scale is not None:
            k = k * self.k_scale.double().cpu().numpy()[None, :, None, None]
            v = v * self.v_scale.double().cpu().numpy()[None, :, None, None]
        scale = self.d ** -0.5 if scale is None else scale
        return oracle.serving.paged_attention(host_f64(self.q.contiguous()), k, v, self.table, self.cu, self.kv, scale,
                                              window)

    def check(self, out, lse, scale=None, window=0, what=""):
        torch.cuda.synchronize()
        ref, rl, mean, size = self.reference(scale, window)
        eight = self.k_scale is not None
        weight = 2 * (self.d + 4) * E * size[..., None] + (2.0 ** -11 if eight else 2.0 ** -8) + (self.max_kv + 64) * E
        half = np.abs(ref) * 2.0 ** -8 if out.dtype == torch.bfloat16 else 0.0
        bound = weight * mean + half + 1e-30
        got, gl = host_f64(out), host_f64(lse)
        err = np.abs(got - ref)
        say(f"  {what}: max err {err.max(initial=0):.3e}, of the bound {np.max(err / bound, initial=0):.2f}")
        assert np.all(np.isfinite(got)), what
        assert np.all(err <= bound), what
        empty = np.isneginf(rl)
        assert np.array_equal(np.isneginf(gl), empty), what
        assert np.all(got[empty] == 0.0), what
        lb = (self.d + 4) * E * size + (self.max_kv + 64) * E + 4 * E * np.abs(np.where(empty, 0, rl))
        assert np.all(np.abs(gl[~empty] - rl[~empty]) <= lb[~empty]), what


SHAPES = [
    # lens, heads_q, heads_kv, d, page, window
    ([(1, 1)], 1, 1, 128, 16, 0),
    ([(1, 1), (0, 0), (1, 17), (0, 9), (1, 64)], 4, 4, 128, 16, 0),
    ([(1, 700), (1, 33), (1, 512), (1, 1)], 10, 2, 128, 64, 0),
    ([(1, 1030)], 40, 8, 128, 16, 0),
    ([(3, 3), (5, 100), (1, 31), (2, 64)], 8, 1, 128, 32, 0),
    ([(9, 500), (4, 4), (1, 320)], 10, 2, 64, 16, 0),
    ([(33, 33), (7, 129), (64, 200)], 4, 4, 64, 128, 0),
    ([(5, 2), (3, 0), (2, 1)], 4, 2, 128, 16, 0),            # tokens before position 0 see nothing
    ([(130, 333), (1, 70), (257, 257)], 6, 2, 128, 32, 0),
    ([(100, 1100)], 5, 1, 64, 1024, 0),
    ([(1, 900), (4, 300), (1, 5)], 8, 2, 128, 16, 1),
    ([(1, 900), (4, 300), (1, 5)], 8, 2, 64, 16, 100),
    ([(150, 400), (40, 40)], 4, 1, 128, 64, 37),
    ([(200, 200), (17, 250)], 2, 2, 64, 16, 5000),
    ([(130, 1333), (1, 700), (257, 957), (0, 30), (300, 1300)], 6, 2, 128, 32, 0),   # many row tiles in one line
    ([(150, 1400), (40, 1040)], 4, 1, 64, 64, 1037),
]


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{len(s[0])}x{max(n for n, _ in s[0])}-{max(k for _, k in s[0])}-"
                                                         f"h{s[1]}.{s[2]}-d{s[3]}-p{s[4]}-w{s[5]}")
def test_attention_matches_oracle(shape, cache):
    lens, hq, hkv, d, page, window = shape
    say(f"attention {shape} {cache}")
    c = Case(lens, hq, hkv, d, page, cache)
    for kind in ("bf16", "f32"):
        out, lse = c.attend(window=window, out_dtype=KIND[kind])
        c.check(out, lse, window=window, what=f"{cache} -> {kind}")
    again, _ = c.attend(window=window, out_dtype=torch.float32)
    assert torch.equal(again, out)


WIDE = [  # at least 256 rows of a key/value head in a sequence, in one part: the kernel for large chunks
    ([(130, 333), (1, 70), (257, 257), (0, 5)], 6, 2, 128, 32, 0),
    ([(100, 1100)], 5, 1, 64, 1024, 0),
    ([(150, 400), (40, 40)], 4, 1, 128, 64, 37),
    ([(300, 64), (64, 300)], 4, 1, 64, 16, 0),
    ([(260, 260), (513, 600)], 2, 2, 128, 16, 0),
    ([(256, 64)], 1, 1, 128, 16, 0),
]


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
@pytest.mark.parametrize("shape", WIDE, ids=lambda s: f"{s[0][0][0]}-{s[0][0][1]}-h{s[1]}.{s[2]}-d{s[3]}-p{s[4]}-w{s[5]}")
def test_attention_of_large_chunks(shape, cache):
    lens, hq, hkv, d, page, window = shape
    say(f"large chunks {shape} {cache}")
    c = Case(lens, hq, hkv, d, page, cache)
    small = torch.empty(16, dtype=torch.uint8, device=DEV)
    out, lse = c.attend(window=window, out_dtype=torch.float32, workspace=small)
    c.check(out, lse, window=window, what="in one part")
    again, al = c.attend(window=window, out_dtype=torch.float32, workspace=small)
    assert torch.equal(again, out) and torch.equal(al, lse)
    for scale in (0.0, -0.7):
        out, lse = c.attend(window=window, out_dtype=torch.bfloat16, workspace=small, scale=scale)
        c.check(out, lse, window=window, scale=scale, what=f"scale {scale}")


def test_attention_of_many_large_chunks():
    """Enough row tiles to fill the GPU: in one part although a workspace is there."""
    c = Case([(300, 300), (5, 900), (290, 700)] * 5, 16, 16, 64, 16, "bf16")
    out, lse = c.attend(out_dtype=torch.float32)
    small = torch.empty(16, dtype=torch.uint8, device=DEV)
    whole, wl = c.attend(out_dtype=torch.float32, workspace=small)
    torch.cuda.synchronize()
    big = torch.arange(c.total, device=DEV) % 595
    big = (big < 300) | (big >= 305)
    assert torch.equal(out[big], whole[big]) and torch.equal(lse[big], wl[big])
    c.check(out, lse, what="many")


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
@pytest.mark.parametrize("n,kv,hq,hkv", [(1, 4000, 4, 2), (6, 3001, 8, 2), (70, 2500, 2, 1)])
def test_attention_split_and_whole(n, kv, hq, hkv, cache):
    """Positions split over workgroups and joined, and in one part (no workspace)."""
    c = Case([(n, kv), (n, kv // 7)], hq, hkv, 128, 64, cache)
    assert tb.tb_paged_attention_workspace(c.q, c.k, c.v, c.table_d, c.cu_d, c.kv_d, c.max_q, c.max_kv) > 0
    say(f"split {n} {kv} {cache}")
    out, lse = c.attend(out_dtype=torch.float32)
    c.check(out, lse, what="split")
    small = torch.empty(16, dtype=torch.uint8, device=DEV)
    whole, wl = c.attend(out_dtype=torch.float32, workspace=small)
    c.check(whole, wl, what="whole")
    # a guess of max_kv that is far off changes nothing but the split
    c.max_kv = 10
    out, lse = c.attend(out_dtype=torch.float32)
    c.max_kv = kv
    c.check(out, lse, what="short guess")


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
@pytest.mark.parametrize("n,kv,whole", [(1, 300, False), (12, 300, False), (150, 300, False), (150, 300, True)])
def test_attention_unseen_values_do_not_reach_a_row(n, kv, whole, cache):
    """NaN and infinities at positions that a token does not see leave it alone;
    at positions that it sees they give what the formula gives."""
    c = Case([(n, kv), (n, n)], 4, 2, 128, 16, cache)
    window = 40
    kw = dict(window=window, out_dtype=torch.float32)
    if whole:
        kw["workspace"] = torch.empty(16, dtype=torch.uint8, device=DEV)
    first, fl = c.attend(**kw)
    c.check(first, fl, window=window, what="clean")
    page_of = lambda x: (int(c.table[0, x // c.page]), x % c.page)  # noqa: E731
    # what lies before every window, and its table entries
    low = kv - n - window
    for x in range(0, low + 1):
        i, s = page_of(x)
        c.k[i, :, s] = float("nan")
        c.v[i, :, :, s] = float("nan")
    c.table[0, :(low + 1) // c.page] = np.where(np.arange((low + 1) // c.page) % 2, 2**31 - 1, -2**31)
    c.ints()
    out, lse = c.attend(**kw)
    torch.cuda.synchronize()
    assert torch.equal(out, first) and torch.equal(lse, fl)
    # a later token's value: the tokens before it are as they were, it and those that see it are not finite there
    for t in sorted({n - 1, n // 2}):
        d = Case([(n, kv), (n, n)], 4, 2, 128, 16, cache)
        i, s = int(d.table[0, (kv - n + t) // 16]), (kv - n + t) % 16
        d.v[i, 1, 3, s] = float("nan") if cache == "fp8" else float("inf")
        d.k[i, 0, s, 5] = float("nan")
        out, lse = d.attend(**kw)
        torch.cuda.synchronize()
        seen = torch.zeros(2 * n, dtype=torch.bool, device=DEV)
        seen[t:min(n, t + window)] = True
        assert torch.equal(out[~seen], first[~seen]), t
        assert torch.isnan(out[seen][:, :2]).all() and torch.isnan(lse[seen][:, :2]).all()    # through the scores
        got = out[seen][:, 2:]
        ok = torch.ones(128, dtype=torch.bool, device=DEV)
        ok[3] = False
        assert torch.equal(lse[seen][:, 2:], fl[seen][:, 2:])
        assert torch.allclose(got[..., ok], first[seen][:, 2:][..., ok], rtol=1e-5, atol=1e-6)
        assert (torch.isnan(got[..., 3]) if cache == "fp8" else got[..., 3] == float("inf")).all()


@pytest.mark.parametrize("cache", ["bf16", "fp8"])
def test_attention_pages_that_are_not_there(cache):
    """Table entries outside the pool: their positions do not exist."""
    c = Case([(2, 200), (20, 90)], 4, 2, 128, 16, cache)
    c.table[0, 3], c.table[0, 12], c.table[1, 0], c.table[1, 2] = -1, c.pages, 2**31 - 1, -2**31
    c.ints()
    out, lse = c.attend(out_dtype=torch.float32)
    c.check(out, lse, what="holes")
    # no page at all, positions past the table, lengths that are negative
    c.table[1, :] = -1
    c.kv = [10**6, 90]
    c.max_kv = 2000
    c.ints()
    out, lse = c.attend(out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert torch.isfinite(out).all() and torch.all(out[2:] == 0) and torch.isneginf(lse[2:]).all()
    c.kv = [-5, 90]
    c.ints()
    out, lse = c.attend(out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert torch.all(out == 0)


def test_attention_rows_of_no_sequence_stay():
    c = Case([(2, 20), (3, 30)], 2, 1, 64, 16, "bf16")
    ref, rl = c.attend(out_dtype=torch.float32)
    out, lse = torch.full((5, 2, 64), 9.0, device=DEV), torch.full((5, 2), 9.0, device=DEV)
    c.cu = [0, 1, 4]
    c.kv = [19, 30]
    c.ints()
    c.attend(out=out, lse=lse)
    torch.cuda.synchronize()
    assert torch.allclose(out[0], ref[0]) and torch.all(out[4] == 9.0) and torch.all(lse[4] == 9.0)
    for cu in ([-4, 1, 99], [3, 1, 0], [2**31 - 1, 0, 2]):   # clamped: nothing outside is read or written
        c.cu = cu
        c.ints()
        out, lse = c.attend(out=torch.zeros(5, 2, 64, device=DEV))
        torch.cuda.synchronize()
        assert torch.isfinite(out).all()


def test_attention_scale_and_large_scores():
    c = Case([(3, 150)], 4, 4, 128, 32, "bf16")
    for scale in (0.0, 2.5, -0.3, 1e-6):
        out, lse = c.attend(scale=scale, out_dtype=torch.float32)
        c.check(out, lse, scale=scale, what=f"scale {scale}")
    c.q.mul_(float("inf"))
    out, _ = c.attend(out_dtype=torch.float32)
    torch.cuda.synchronize()
    assert torch.isnan(out).all()       # inf - inf in every score


def test_attention_on_a_stream_and_in_a_graph():
    c = Case([(1, 3000), (2, 800)], 8, 2, 128, 64, "bf16")
    ref, rl = c.attend()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out, lse = c.attend(stream=s)
    s.synchronize()
    assert torch.equal(out, ref) and torch.equal(lse, rl)
    ws = torch.empty(tb.tb_paged_attention_workspace(c.q, c.k, c.v, c.table_d, c.cu_d, c.kv_d, c.max_q, c.max_kv),
                     dtype=torch.uint8, device=DEV)
    out, lse = torch.empty_like(ref), torch.empty_like(rl)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.append()
        c.attend(out=out, lse=lse, workspace=ws)
    for _ in range(3):
        c.q.normal_()
        c.new_k.normal_()
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        e, el = c.attend()
        assert torch.equal(out, e) and torch.equal(lse, el)


def test_cache_past_32_bit_offsets():
    """Pages past 2^31 elements of the pool."""
    pages, hkv, page, d = 17000, 8, 128, 128
    assert pages * hkv * page * d > 2**31
    k = torch.empty(pages, hkv, page, d, dtype=torch.bfloat16, device=DEV)
    v = torch.empty(pages, hkv, d, page, dtype=torch.bfloat16, device=DEV)
    c = Case([(3, 600)], 8, hkv, d, page, "bf16", poison=False)
    table = pages - 1 - 2 * np.arange(c.table.shape[1])
    for x in range(5):
        k[int(table[x])] = c.k[int(c.table[0, x])]
        v[int(table[x])] = c.v[int(c.table[0, x])]
    c.append()
    ref, rl = c.attend()
    c.k, c.v = k, v
    c.table[0] = table
    c.ints()
    c.append()
    out, lse = c.attend()
    torch.cuda.synchronize()
    assert torch.equal(out, ref) and torch.equal(lse, rl)


# ------------------------------------------------------------------ append

@pytest.mark.parametrize("cache", ["bf16", "fp8"])
@pytest.mark.parametrize("lens,hkv,d,page", [
    ([(1, 1), (1, 100), (0, 50), (1, 16)], 2, 128, 16),
    ([(70, 70), (3, 130), (129, 300)], 3, 64, 32),
    ([(64, 64), (100, 1000)], 1, 128, 1024),
    ([(5, 2), (4, 0), (1, 33)], 2, 64, 16),                 # tokens before position 0
    ([(300, 300)], 8, 128, 128),
])
def test_append(lens, hkv, d, page, cache):
    say(f"append {lens} {hkv} {d} {page} {cache}")
    c = Case(lens, 1, hkv, d, page, cache, poison=False)
    if cache == "fp8" and c.total:
        c.new_k[0, 0, :4] = torch.tensor([float("nan"), 1e9, -1e9, 0.0], device=DEV)
        c.new_v[c.total - 1, hkv - 1, :2] = torch.tensor([float("inf"), -float("inf")], device=DEV)
    c.table[0, 0] = -1 if len(lens) > 3 else c.table[0, 0]   # a page that is not there
    c.ints()
    bits = torch.uint8 if cache == "fp8" else torch.int16
    k, v = c.k.clone().view(bits).cpu(), c.v.clone().view(bits).cpu()

    def code(x, scale, h):
        if cache == "bf16":
            return x.cpu().view(bits)
        return (x.float() / scale[h]).clamp(-448, 448).to(torch.float8_e4m3fn).cpu().view(bits)

    for b in range(len(lens)):
        for r, pos in oracle.serving.paged_rows(c.cu, c.kv, b):
            at = oracle.serving.paged_slot(c.table, page, c.pages, b, pos)
            if at is None:
                continue
            for h in range(hkv):
                k[at[0], h, at[1]] = code(c.new_k[r, h], c.k_scale, h)
                v[at[0], h, :, at[1]] = code(c.new_v[r, h], c.v_scale, h)
    c.append()
    torch.cuda.synchronize()
    gk, gv = c.k.view(bits).cpu(), c.v.view(bits).cpu()
    if cache == "fp8":   # the sign of a NaN is not fixed
        for g, w in ((gk, k), (gv, v)):
            nan = (w & 0x7f) == 0x7f
            assert torch.equal((g & 0x7f) == 0x7f, nan)
            g[nan] = w[nan]
    assert torch.equal(gk, k) and torch.equal(gv, v)


def test_append_every_value():
    """All bf16 patterns over the scales of eight heads, each pattern with each
    scale: the codes are those of the division, bit for bit."""
    c = Case([(64, 64)], 8, 8, 128, 16, "fp8", poison=False)
    every = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).to(DEV)
    scales = torch.tensor([1.0, 0.0371, 2.0 / 3, 1e-30, 7e25, 1.7e-12, 449.0, 3e-3], device=DEV)
    for i in range(8):
        say(f"append every value, turn {i}")
        c.new_k, c.new_v = every.view(64, 8, 128), every.flip(0).view(64, 8, 128)
        c.k_scale, c.v_scale = scales.roll(i).contiguous(), scales.roll(i + 3).contiguous()
        c.append()
        torch.cuda.synchronize()
        pages = torch.from_numpy(c.table[0, :4]).to(DEV)
        k = c.k[pages].view(torch.uint8).permute(0, 2, 1, 3).reshape(64, 8, 128)
        v = c.v[pages].view(torch.uint8).permute(0, 3, 1, 2).reshape(64, 8, 128)
        for got, x, scale in ((k, c.new_k, c.k_scale), (v, c.new_v, c.v_scale)):
            want = (x.float() / scale[:, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            nan = torch.isnan(x)
            assert ((got & 0x7f) == 0x7f)[nan].all()
            assert torch.equal(got[~nan], want[~nan])


def test_append_then_attend():
    """Chunk by chunk through the cache is the whole sequence at once."""
    c = Case([(200, 200)], 4, 2, 128, 32, "bf16", poison=False)
    c.append()
    whole, wl = c.attend(out_dtype=torch.float32)
    c.check(whole, wl, what="whole")
    q, nk, nv = c.q, c.new_k, c.new_v
    c.k.fill_(float("nan"))
    c.v.fill_(float("nan"))
    at = 0
    for n in (1, 7, 64, 1, 90, 37):
        c.q, c.new_k, c.new_v = q[at:at + n], nk[at:at + n], nv[at:at + n]
        at += n
        c.cu, c.kv, c.max_q, c.max_kv = [0, n], [at], n, at
        c.ints()
        c.append()
        out, lse = c.attend(out_dtype=torch.float32)
        torch.cuda.synchronize()
        # each is within the bounds of the oracle; two of them within twice
        assert torch.allclose(out, whole[at - n:at], rtol=0, atol=2 * 2.0 ** -8 * 4)
        assert torch.allclose(lse, wl[at - n:at], rtol=1e-5, atol=1e-4)


def test_binding_refuses_shapes_and_dtypes():
    c = Case([(2, 20)], 2, 1, 64, 16, "bf16")
    ok = dict(q=c.q, k_cache=c.k, v_cache=c.v, block_table=c.table_d, cu_q=c.cu_d, kv_len=c.kv_d, max_q=2, max_kv=20)
    tb.tb_paged_attention(**ok)
    for bad, err in ((dict(q=c.q.float()), ValueError), (dict(q=c.q[:, :, ::2]), ValueError),
                     (dict(v_cache=c.k), ValueError), (dict(k_cache=c.k.float(), v_cache=c.v.float()), TypeError),
                     (dict(block_table=c.table_d.long()), TypeError), (dict(kv_len=c.kv_d[:0]), ValueError),
                     (dict(out=torch.empty(1, device=DEV)), ValueError), (dict(window=-1), tb.TBError),
                     (dict(scale=float("inf")), tb.TBError), (dict(out=c.q.contiguous()[:, :, :32]), ValueError),
                     (dict(k_scale=torch.ones(1, device=DEV)), ValueError), (dict(lse=torch.empty(2, 3, device=DEV)), ValueError)):
        with pytest.raises(err):
            tb.tb_paged_attention(**{**ok, **bad})
    with pytest.raises(ValueError):
        tb.tb_paged_append(c.new_k, c.new_v[:1], c.k, c.v, c.table_d, c.cu_d, c.kv_d, 2)
    with pytest.raises(ValueError):
        tb.tb_paged_append(c.new_k.transpose(0, 1).contiguous().transpose(0, 1), c.new_v, c.k, c.v, c.table_d, c.cu_d[:1],
                           c.kv_d, 2)

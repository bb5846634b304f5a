"""More operators of a serving step, as cases to be measured.

Between a projection and the verification of drafts, a decoder with rotary
positions and a small cache needs: the position rotation of queries and keys on
their way out and into the cache, a cache of 4-bit codes with the attention that
reads it and a way to read it back, and the probabilities of tokens from logits
(penalties, biases, grammar masks, temperature).  `run` computes one call of one
of them, in elementary torch operations where `own` is false and by the library's
entry points where it is true.

Sizes: 5120 channels as 40 heads of 128 and batches up to 16 are the decoder
layer of this repository's benchmark; 8 key/value heads, chunks, page sizes,
lengths and vocabularies are those of the serving operators' cases.
"""

import math
import random

import numpy as np
import torch

own = False

BASE = 500000.0


# ------------------------------------------------------------------- cases

def _rotary(name, b, chunk, kv, hq, hkv, d, rot, pairs, page, cache, turn, factor, ragged):
    return {"name": name, "op": "rotary", "b": b, "chunk": chunk, "kv": kv, "hq": hq, "hkv": hkv, "d": d, "rot": rot,
            "pairs": pairs, "page": page, "cache": cache, "turn": turn, "factor": factor, "ragged": ragged}


def _attn(name, b, chunk, kv, hq, hkv, d, page, window, ragged):
    return {"name": name, "op": "attention", "b": b, "chunk": chunk, "kv": kv, "hq": hq, "hkv": hkv, "d": d,
            "page": page, "window": window, "ragged": ragged}


def _probs(name, b, drafts, vocab, kind, history, bias, grammar):
    return {"name": name, "op": "probs", "b": b, "drafts": drafts, "vocab": vocab, "kind": kind, "history": history,
            "bias": bias, "grammar": grammar}


def listed():
    return [
        # one user's next token: latency
        _rotary("rotary-step-1", 1, 1, 1000, 40, 8, 128, 128, "halves", 16, "bf16", False, 1.0, False),
        # a decode batch in the rotated basis of the products, kept in it, into 4 bits; then the cache read back
        _rotary("rotary-step-16-int4", 16, 1, 256, 40, 8, 128, 128, "halves", 16, "int4", True, 1.0, True),
        # prompt chunks, positions on part of each head, neighbours paired, scaled for a long context, an 8-bit cache
        _rotary("rotary-chunk-fp8", 4, 2048, 2500, 40, 8, 128, 64, "neighbours", 64, "fp8", False, 1.2, True),
        # prompt chunks into 4 bits; then the cache read back
        _rotary("rotary-chunk-int4", 4, 2048, 2500, 40, 8, 128, 128, "halves", 64, "int4", True, 1.0, True),
        # one user's next token, a key/value head for each query head, small pages: latency
        _attn("attention4-step-1", 1, 1, 1000, 40, 40, 128, 16, 0, False),
        # a full decode batch at mixed lengths, shared heads
        _attn("attention4-step-16", 16, 1, 8192, 40, 8, 128, 64, 0, True),
        # few users with long contexts
        _attn("attention4-step-long", 4, 1, 65536, 40, 8, 128, 64, 0, True),
        # chunks of prompts over what is cached of them
        _attn("attention4-chunk", 4, 2048, 8192, 40, 8, 128, 64, 0, True),
        # a sliding window, odd lengths, 64-wide heads, small pages
        _attn("attention4-chunk-window", 2, 777, 6000, 16, 16, 64, 16, 1000, False),
        # one user's next token, a small odd vocabulary
        _probs("probs-1", 1, 0, 32003, "fp32", 300, 20, False),
        # few users' drafted tokens under a grammar, long histories, a large odd vocabulary
        _probs("probs-draft-8", 8, 8, 131073, "bf16", 4000, 0, True),
        # a batch of drafts
        _probs("probs-draft-32", 32, 8, 131073, "fp32", 2000, 100, False),
    ]


def _log(rng, lo, hi):
    """A whole number from lo to hi, even over its logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def _drawn(rng):
    op = rng.choice(["rotary", "rotary", "attention", "attention", "probs"])
    page, d = rng.choice([16, 32, 64, 128]), rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8, 8, 10, 40])
    group = rng.choice([1, 2, 4, 5, 8]) if hkv <= 8 else 1
    if op == "rotary":
        chunk = rng.choice([1, _log(rng, 1, 2048)])
        c = _rotary("", _log(rng, 1, 16), chunk, max(chunk, _log(rng, 1, 2500)), hkv * group, hkv, d,
                    rng.choice([d, 16 * rng.randint(1, d // 16)]), rng.choice(["halves", "neighbours"]), page,
                    rng.choice(["bf16", "fp8", "int4"]), d == 128 and rng.random() < 0.5, rng.choice([1.0, 1.2]),
                    rng.random() < 0.6)
    elif op == "attention":
        chunk = rng.choice([1, _log(rng, 1, 16), _log(rng, 1, 2048)])
        kv = max(chunk, _log(rng, 1, 65536 if chunk <= 16 else 8192))
        c = _attn("", _log(rng, 1, 16), chunk, kv, hkv * group, hkv, d, page, rng.choice([0, 0, _log(rng, 1, 4096)]),
                  rng.random() < 0.6)
    else:
        c = _probs("", _log(rng, 1, 32), rng.choice([0, rng.randint(1, 8)]), _log(rng, 500, 131073),
                   rng.choice(["fp32", "bf16"]), _log(rng, 1, 4000), rng.choice([0, _log(rng, 1, 300)]),
                   rng.random() < 0.4)
    del c["name"]
    return c


def draw(rng):
    tops = {}
    for c in listed():
        w = work(c)
        t = tops.setdefault(c["op"], [0.0, 0.0])
        t[0], t[1] = max(t[0], w["bytes"]), max(t[1], w["flops"])
    while True:
        c = _drawn(rng)
        w, t = work(c), tops[c["op"]]
        # the cache, and the rectangle that a window leaves most of unseen, are held to the listed cases' too
        room = c["op"] == "probs" or c["b"] * c["kv"] * c["hkv"] * c["d"] <= 1 << 28
        if c["op"] == "attention":
            room = room and c["b"] * c["hq"] * c["chunk"] * c["kv"] <= 4 * 40 * 2048 * 8192
        if room and w["bytes"] <= t[0] and w["flops"] <= t[1]:
            return c


def _lengths(c):
    """New tokens and cached tokens (the new ones among them) of each sequence: by the case alone."""
    r = random.Random("%(b)d %(chunk)d %(kv)d" % c)
    n, kv = [], []
    for i in range(c["b"]):
        n.append(c["chunk"] if not c["ragged"] or i == 0 else r.randint(1, c["chunk"]))
        kv.append(c["kv"] if not c["ragged"] or i == 0 else r.randint(max(n[i], c["kv"] // 4), c["kv"]))
    return n, kv


def _token_lengths(c):
    """Drafts, history and prompt tokens of each sequence: by the case alone."""
    r = random.Random("%(b)d %(drafts)d %(vocab)d %(history)d" % c)
    n = [c["drafts"]] + [r.randint(0, c["drafts"]) for _ in range(c["b"] - 1)]
    h = [c["history"]] + [r.randint(0, c["history"]) for _ in range(c["b"] - 1)]
    return n, h, [r.randint(0, x) for x in h]


# ------------------------------------------------------------------ inputs

_KIND = {"bf16": torch.bfloat16, "fp32": torch.float32, "fp8": torch.float8_e4m3fn}


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _offsets(n):
    cu = [0]
    for x in n:
        cu.append(cu[-1] + x)
    return cu


def _pages(c, kv, seed):
    """Each sequence's pages, scattered over the pool as a serving program hands them out."""
    per = [-(-x // c["page"]) for x in kv]
    ids = list(range(sum(per)))
    random.Random(seed).shuffle(ids)
    table, at, width = [], 0, -(-c["kv"] // c["page"])
    for m in per:
        table.append(ids[at:at + m] + [0] * (width - m))
        at += m
    return table, sum(per)


def _codes4(shape, g):
    """4-bit codes as those of normal values between their least and their largest: few at the ends."""
    x = torch.empty(shape, dtype=torch.uint8, device="cuda")
    for i in range(0, shape[0], 256):  # a part of the pool at a time
        part = x[i:i + 256]
        n = torch.randn((2,) + tuple(part.shape), generator=g, device="cuda") * 2.8 + 7.5
        n = n.round_().clamp_(0, 15).to(torch.uint8)
        part.copy_(n[0] | (n[1] << 4))
    return x


def _cached(c, kind, seed):
    n, kv = _lengths(c)
    g = _gen(seed)
    table, pages = _pages(c, kv, seed)
    s = {"op": c["op"], "n": n, "kv": kv, "max_q": max(n), "max_kv": max(kv), "page": c["page"], "d": c["d"]}
    s["cu"], s["kv_len"], s["table"] = _ints(_offsets(n)), _ints(kv), _ints(table)
    s["k_scale"] = s["v_scale"] = None
    hkv, page, d = c["hkv"], c["page"], c["d"]
    if kind == "int4":
        s["k_cache"], s["v_cache"] = _codes4((pages, hkv, page, d // 2), g), _codes4((pages, hkv, d // 2, page), g)
        # steps and offsets of normal values; the offset is the value of code -64
        for which, at in (("k", 3), ("v", 2)):
            step = 0.3 + 0.1 * torch.rand((pages, hkv, page), generator=g, device="cuda")
            low = -2.6 + 0.4 * torch.randn((pages, hkv, page), generator=g, device="cuda")
            step = step.half()
            s[which + "_scale"] = torch.stack([step, (low - 64 * step.float()).half()], at).contiguous()
        return s, g
    k = torch.randn((pages, hkv, page, d), generator=g, device="cuda", dtype=torch.bfloat16)
    v = torch.randn((pages, hkv, d, page), generator=g, device="cuda", dtype=torch.bfloat16)
    if kind == "fp8":
        # a head's scale puts its values in the middle of e4m3's range
        k, v = k * 8, v * 8
        s["k_scale"] = (0.1 + 0.05 * torch.rand(hkv, generator=g, device="cuda"))
        s["v_scale"] = (0.1 + 0.05 * torch.rand(hkv, generator=g, device="cuda"))
    s["k_cache"], s["v_cache"] = k.to(_KIND[kind]), v.to(_KIND[kind])
    return s, g


def _frequencies(rot):
    """Rotations of a pair for a step of one position, in radians."""
    return (BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)).to(torch.float32).cuda()


def _hadamard(dtype):
    h = torch.ones(1, 1, dtype=dtype, device="cuda")
    while h.shape[0] < 128:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h / math.sqrt(128.0)


def prepare(case, seed):
    c = case
    if c["op"] == "attention":
        s, g = _cached(c, "int4", seed)
        fused = torch.randn((sum(s["n"]), c["hq"] + 2 * c["hkv"], c["d"]), generator=g, device="cuda").to(torch.bfloat16)
        s["q"] = fused[:, :c["hq"]]
        s["scale"], s["window"] = 1.5 / math.sqrt(c["d"]), c["window"]
        return s
    if c["op"] == "rotary":
        s, g = _cached(c, c["cache"], seed)
        fused = torch.randn((sum(s["n"]), c["hq"] + 2 * c["hkv"], c["d"]), generator=g, device="cuda").to(torch.bfloat16)
        s["q"], s["k"], s["v"] = fused.split([c["hq"], c["hkv"], c["hkv"]], dim=1)
        s["freq"], s["factor"] = _frequencies(c["rot"]), c["factor"]
        s["neighbours"], s["turn"] = c["pairs"] == "neighbours", c["turn"]
        s["hadamard"] = _hadamard(torch.float64)
        if c["cache"] == "int4":
            s["cu_all"], s["total"] = _ints(_offsets(s["kv"])), sum(s["kv"])
        return s
    g = _gen(seed)
    n, h, prompt = _token_lengths(c)
    rows, v = sum(n) + c["b"], c["vocab"]
    # tokens that a model likes, for the whole batch and for each row
    liked = torch.randn(v, generator=g, device="cuda") * 1.5
    logits = (liked + torch.randn((rows, v), generator=g, device="cuda") * 2.0).to(_KIND[c["kind"]])
    p = torch.softmax(liked * 2, 0)

    def tokens(m):
        return torch.multinomial(p, m, True, generator=g).to(torch.int32) if m else _ints([])

    s = {"op": "probs", "logits": logits, "n": n, "max_draft": max(n), "cu": _ints(_offsets(n)), "drafts": tokens(sum(n)),
         "history": tokens(sum(h)), "cu_history": _ints(_offsets(h)), "prompt": _ints(prompt)}
    # temperature (a greedy sequence among them), penalties of repeats, of presence, of frequency
    each = torch.rand((c["b"], 4), generator=g, device="cuda")
    s["params"] = torch.stack([0.5 + each[:, 0], 1 + 0.3 * each[:, 1], each[:, 2], 0.5 * each[:, 3]], 1).contiguous()
    if c["b"] > 3:
        s["params"][3, 0] = 0.0
    s["bias"] = None
    if c["bias"]:
        many = [c["bias"]] + [random.Random(i).randint(0, c["bias"]) for i in range(1, c["b"])]
        many = [min(m, v) for m in many]
        ids = [torch.randperm(v, generator=g, device="cuda")[:m] for m in many]
        s["bias"] = (torch.cat(ids).to(torch.int32), torch.randn(sum(many), generator=g, device="cuda") * 3,
                     _ints(_offsets(many)))
    s["mask"] = s["mask_row"] = None
    if c["grammar"]:
        # a mask for most rows: of few tokens, or of many
        words = -(-v // 32)
        s["mask_row"] = _ints([-1 if i % 4 == 3 else i // 4 * 3 + i % 4 for i in range(rows)])
        masks = (rows - 1) // 4 * 3 + min((rows - 1) % 4 + 1, 3)
        s["mask"] = torch.empty((masks, words), dtype=torch.int32, device="cuda")
        for i in range(masks):
            share = 0.5 if i % 2 else 0.01
            allowed = torch.rand((words, 32), generator=g, device="cuda") < share
            bits = (allowed.long() << torch.arange(32, device="cuda")).sum(1)
            s["mask"][i] = torch.where(bits >= 1 << 31, bits - (1 << 32), bits).to(torch.int32)
    return s


# ------------------------------------------------------------ plain forms

def _positions(s, length):
    """Page and slot of each sequence's positions 0 .. length - 1, and which of them are cached."""
    pos = torch.arange(length, device="cuda")
    live = pos[None] < s["kv_len"][:, None]
    page = torch.where(live, s["table"].long()[:, pos // s["page"]], 0)
    return page, (pos % s["page"])[None].expand_as(page), live


def _owners(s):
    """Sequence of each new token, its place in the sequence's chunk, and its position."""
    cu = s["cu"].long()
    at = torch.arange(sum(s["n"]), device="cuda")
    b = torch.searchsorted(cu[1:], at, right=True)
    j = at - cu[b]
    return b, j, s["kv_len"].long()[b] - (cu[b + 1] - cu[b]) + j


def _values4(codes, scale, offset):
    """Values of channels 8 g + i and 8 g + i + 4 in byte 4 g + i (last axis)."""
    x = codes.view(codes.shape[:-1] + (-1, 1, 4))
    n = torch.cat([x & 15, x >> 4], -2).reshape(codes.shape[:-1] + (-1,))
    # the product has 18 bits; the sum has few enough more for 32
    return torch.addcmul(offset.float()[..., None], scale.float()[..., None], n.float() + 64).half().float()


def _cached_values(s, page, slot):
    """Keys and values of these places, [places .., heads, d]."""
    k = _values4(s["k_cache"][page, :, slot], s["k_scale"][page, :, slot, 0], s["k_scale"][page, :, slot, 1])
    v = _values4(s["v_cache"][page, :, :, slot], s["v_scale"][page, :, 0, slot], s["v_scale"][page, :, 1, slot])
    return k, v


def _plain_attention(s):
    tokens, hq, d = s["q"].shape
    hkv = s["k_cache"].shape[1]
    group, nb, nq, nk = hq // hkv, s["kv_len"].shape[0], s["max_q"], s["max_kv"]
    page, slot, live = _positions(s, nk)
    k, v = _cached_values(s, page, slot)                                   # [B, L, Hkv, D]
    b, j, pos = _owners(s)
    q = torch.zeros((nb, nq, hq, d), device="cuda")
    q[b, j] = s["q"].float()
    at = torch.full((nb, nq), -1, dtype=torch.int64, device="cuda")
    at[b, j] = pos
    q = q.view(nb, nq, hkv, group, d).permute(0, 2, 3, 1, 4).reshape(nb * hkv, group * nq, d)
    k = k.permute(0, 2, 3, 1).reshape(nb * hkv, d, nk).contiguous()
    v = v.permute(0, 2, 1, 3).reshape(nb * hkv, nk, d).contiguous()
    key = torch.arange(nk, device="cuda")
    seen = key[None, None] <= at[:, :, None]
    if s["window"]:
        seen &= key[None, None] > at[:, :, None] - s["window"]
    scores = torch.bmm(q, k).view(nb, hkv, group, nq, nk) * s["scale"]
    scores = scores.masked_fill(~seen[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    e = torch.exp(scores - top)
    total = e.sum(-1, keepdim=True)
    o = torch.bmm(e.view(nb * hkv, group * nq, nk), v).view(nb, hkv, group, nq, d)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (top + torch.log(total))[..., 0]
    o = o.permute(0, 3, 1, 2, 4).reshape(nb, nq, hq, d)[b, j]
    lse = lse.permute(0, 3, 1, 2).reshape(nb, nq, hq)[b, j]
    return {"out": o.to(torch.bfloat16), "lse": lse}


def _nearest_half(x):
    """The nearest fp16 of 64-bit values (a conversion would round to 32 bits first)."""
    step = torch.exp2((torch.frexp(x)[1] - 11).clamp(min=-24).double())
    return (torch.round(x / step) * step).half()


def _quantised4(x):
    """Codes of 64-bit rows, and their scales and offsets."""
    x = x.clamp(-4096.0, 4096.0)
    low, high = x.amin(-1), x.amax(-1)
    scale = _nearest_half((high - low) / 15)
    offset = _nearest_half(low - 64 * scale.double())
    n = (torch.round((x - offset.double()[..., None]) / scale.double()[..., None]) - 64).clamp(0, 15)
    n = torch.where(scale[..., None] > 0, n, 0.0).to(torch.uint8)
    n = n.view(n.shape[:-1] + (-1, 2, 4))
    return (n[..., 0, :] | (n[..., 1, :] << 4)).flatten(-2), scale, offset


def _plain_rotary(s):
    b, _, pos = _owners(s)
    page, slot = s["table"].long()[b, pos // s["page"]], pos % s["page"]
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    if s["turn"]:
        q, k, v = q @ s["hadamard"], k @ s["hadamard"], v @ s["hadamard"]
    # angles of far positions need 64 bits
    angle = pos.double()[:, None] * s["freq"].double()[None]
    cos, sin = (torch.cos(angle) * s["factor"])[:, None], (torch.sin(angle) * s["factor"])[:, None]
    half = s["freq"].shape[0]

    def rotated(x):
        r, rest = x[..., :2 * half], x[..., 2 * half:]
        x0, x1 = (r[..., 0::2], r[..., 1::2]) if s["neighbours"] else (r[..., :half], r[..., half:])
        y0, y1 = x0 * cos - x1 * sin, x0 * sin + x1 * cos
        y = torch.stack([y0, y1], -1).flatten(-2) if s["neighbours"] else torch.cat([y0, y1], -1)
        return torch.cat([y, rest], -1)

    q, k = rotated(q), rotated(k)
    if s["turn"]:
        q, k = q @ s["hadamard"], k @ s["hadamard"]
    q = q.to(torch.bfloat16)
    if s["k_cache"].dtype == torch.uint8:
        codes, scale, offset = _quantised4(k)
        s["k_cache"][page, :, slot], s["k_scale"][page, :, slot] = codes, torch.stack([scale, offset], -1)
        codes, scale, offset = _quantised4(v)
        s["v_cache"][page, :, :, slot], s["v_scale"][page, :, :, slot] = codes, torch.stack([scale, offset], -1)
        page, slot, live = _positions(s, s["max_kv"])
        k, v = _cached_values(s, page[live], slot[live])
        return {"q": q, "k": k, "v": v}
    kind, as_bits = s["k_cache"].dtype, torch.int16
    if s["k_scale"] is not None:
        as_bits = torch.uint8
        k = (k / s["k_scale"].double()[None, :, None]).clamp(-448.0, 448.0)
        v = (v / s["v_scale"].double()[None, :, None]).clamp(-448.0, 448.0)
    s["k_cache"].view(as_bits)[page, :, slot] = k.to(kind).view(as_bits)
    s["v_cache"].view(as_bits)[page, :, :, slot] = v.to(kind).view(as_bits)
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_probs(s):
    logits, cu, v = s["logits"], s["cu"].long(), s["logits"].shape[1]
    nb, rows = cu.shape[0] - 1, logits.shape[0]
    row = torch.arange(rows, device="cuda")
    first = cu[:-1] + torch.arange(nb, device="cuda")
    seq = torch.searchsorted(first, row, right=True) - 1
    x = logits.float()
    if s["bias"] is not None:
        ids, values, cu_bias = s["bias"]
        owner = torch.searchsorted(cu_bias[1:].long(), torch.arange(ids.shape[0], device="cuda"), right=True)
        bias = torch.zeros((nb, v), device="cuda")
        bias[owner, ids.long()] = values
        x = x + bias[seq]
    # tokens of the prompt are only repeated, those since then also counted
    at = torch.arange(s["history"].shape[0], device="cuda")
    cu_h = s["cu_history"].long()
    owner = torch.searchsorted(cu_h[1:], at, right=True)
    made = at - cu_h[owner] >= s["prompt"].long()[owner]
    count = torch.zeros((2, nb, v), dtype=torch.int32, device="cuda")
    count.index_put_((made.long(), owner, s["history"].long()), torch.ones_like(at, dtype=torch.int32), accumulate=True)
    prompt, count = count[0][seq] > 0, count[1][seq]
    # a row's drafts before it
    for j in range(s["max_draft"]):
        later = torch.nonzero(row - first[seq] > j)[:, 0]
        count[later, s["drafts"].long()[cu[seq[later]] + j]] += 1
    t, repeats, presence, frequency = s["params"][seq].unbind(1)
    seen = prompt | (count > 0)
    x = torch.where(seen, torch.where(x > 0, x / repeats[:, None], x * repeats[:, None]), x)
    x = x - (frequency[:, None] * count + presence[:, None] * (count > 0))
    if s["mask"] is not None:
        bit = torch.arange(v, device="cuda")
        allowed = (s["mask"][:, bit // 32] >> (bit % 32)) & 1
        none = s["mask_row"] < 0
        allowed = torch.where(none[:, None], 1, allowed[s["mask_row"].long().clamp(min=0)])
        x = x.masked_fill(allowed == 0, -math.inf)
    top = x.amax(1, keepdim=True)
    e = torch.exp((x - torch.where(top == -math.inf, 0.0, top)) / torch.where(t > 0, t, 1.0)[:, None])
    total = e.sum(1, keepdim=True)
    p = torch.where(total > 0, e / total, 0.0)
    hot = torch.zeros_like(p)
    hot.scatter_(1, torch.argmax((x == top).to(torch.uint8), 1, keepdim=True), (top > -math.inf).float())
    return {"p": torch.where((t > 0)[:, None], p, hot)}


# -------------------------------------------------------------------- run

def run(state):
    s = state
    if not own:
        return {"attention": _plain_attention, "rotary": _plain_rotary, "probs": _plain_probs}[s["op"]](s)
    from ternary_weights_hadamard_amd import tb
    if s["op"] == "attention":
        out, lse = tb.tb_paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["cu"], s["kv_len"],
                                         s["max_q"], s["max_kv"], scale=s["scale"], window=s["window"],
                                         k_scale=s["k_scale"], v_scale=s["v_scale"], with_lse=True)
        return {"out": out, "lse": lse}
    if s["op"] == "rotary":
        q = tb.tb_paged_append_rotary(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["cu"], s["kv_len"],
                                      s["max_q"], s["freq"], factor=s["factor"], neighbours=s["neighbours"],
                                      turn_in=s["turn"], turn_out=s["turn"], turn_v=s["turn"], k_scale=s["k_scale"],
                                      v_scale=s["v_scale"])
        if s["k_cache"].dtype != torch.uint8:
            return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        k, v = tb.tb_paged_read(s["k_cache"], s["v_cache"], s["table"], s["cu_all"], s["kv_len"], s["total"], s["max_kv"],
                                k_scale=s["k_scale"], v_scale=s["v_scale"], out_dtype=torch.float32)
        return {"q": q, "k": k, "v": v}
    return {"p": tb.tb_token_probs(s["logits"], s["params"], s["drafts"], s["cu"], s["max_draft"], history=s["history"],
                                   cu_history=s["cu_history"], prompt_len=s["prompt"], bias=s["bias"], mask=s["mask"],
                                   mask_row=s["mask_row"])}


def work(case):
    c = case
    if c["op"] == "probs":
        n, h, _ = _token_lengths(c)
        rows = sum(n) + c["b"]
        each = 4 + (2 if c["kind"] == "bf16" else 4)
        return {"bytes": rows * c["vocab"] * (each + (0.75 / 8 if c["grammar"] else 0)) + 4.0 * sum(h) + 8.0 * c["b"] * c["bias"],
                "flops": 6.0 * rows * c["vocab"]}
    n, kv = _lengths(c)
    row, tokens = c["hkv"] * c["d"], sum(n)
    cached = {"bf16": 2.0, "fp8": 1.0, "int4": 0.5 + 4.0 / c["d"]}[c.get("cache", "int4")]  # bytes of a value
    if c["op"] == "rotary":
        moved = tokens * (4.0 * c["hq"] * c["d"] + 2 * row * (2 + cached))
        if c["cache"] == "int4":
            moved += sum(kv) * 2 * row * (4 + cached)
        turned = 14 * (3 * c["hkv"] + 2 * c["hq"]) if c["turn"] else 0
        return {"bytes": moved, "flops": tokens * (3.0 * (c["hq"] + c["hkv"]) * c["rot"] + turned * c["d"])}
    keys, pairs = 0, 0
    for m, have in zip(n, kv):
        w = c["window"] or have
        keys += min(have, w + m - 1)
        # the token at position x sees min(x + 1, w) keys
        first = have - m
        short = max(0, min(m, w - first))
        pairs += short * (first + 1) + short * (short - 1) // 2 + (m - short) * w
    return {"bytes": 2.0 * keys * row * cached + tokens * c["hq"] * (4.0 * c["d"] + 4), "flops": 4.0 * c["d"] * c["hq"] * pairs}


# ------------------------------------------------------------------ exact

def exact(case, seed):
    """The definitions, sequence by sequence, in 64 bits."""
    c, s = case, prepare(case, seed)
    return {"attention": _exact_attention, "rotary": _exact_rotary, "probs": _exact_probs}[c["op"]](c, s)


def _exact_cached(s, b, have):
    """Keys and values of a sequence's first positions in 64 bits, [position, head, channel]."""
    ids = s["table"][b, :-(-have // s["page"])].long()

    def of(codes, scale, offset):  # [position, head, byte], [position, head]
        out = torch.empty(codes.shape[:2] + (s["d"],), dtype=torch.float64, device="cuda")
        for i in range(4):
            for high in range(2):
                n = (codes[..., i::4] // 16 if high else codes[..., i::4] % 16).double()
                out[..., i + 4 * high::8] = (64 + n) * scale.double()[..., None] + offset.double()[..., None]
        return out.float().half().double()  # exact in 32 bits: a scale's 11 bits times 7, beside the offset

    k = s["k_cache"][ids].transpose(1, 2).flatten(0, 1)[:have]
    v = s["v_cache"][ids].permute(0, 3, 1, 2).flatten(0, 1)[:have]
    ks = s["k_scale"][ids].transpose(1, 2).flatten(0, 1)[:have]
    vs = s["v_scale"][ids].permute(0, 3, 1, 2).flatten(0, 1)[:have]
    return of(k, ks[..., 0], ks[..., 1]), of(v, vs[..., 0], vs[..., 1])


def _exact_attention(c, s):
    n, kv = _lengths(c)
    group, outs, lses, first = c["hq"] // c["hkv"], [], [], 0
    for b, (m, have) in enumerate(zip(n, kv)):
        k, v = _exact_cached(s, b, have)
        pos = torch.arange(have - m, have, device="cuda")[:, None]
        key = torch.arange(have, device="cuda")[None]
        hide = (key > pos) | ((key <= pos - c["window"]) if c["window"] else torch.zeros_like(key, dtype=torch.bool))
        out = torch.empty((m, c["hq"], c["d"]), dtype=torch.float64, device="cuda")
        lse = torch.empty((m, c["hq"]), dtype=torch.float64, device="cuda")
        for h in range(c["hq"]):
            kh, vh = k[:, h // group], v[:, h // group]
            x = (s["q"][first:first + m, h].double() @ kh.T.contiguous()) * s["scale"]
            x[hide] = -math.inf
            lse[:, h] = torch.logsumexp(x, 1)
            out[:, h] = torch.exp(x - lse[:, h, None]) @ vh
        outs.append(out)
        lses.append(lse)
        first += m
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def _butterflies(x):
    shape, x = x.shape, x.reshape(-1, 128)
    for bit in range(7):
        y = x.view(-1, 128 >> (bit + 1), 2, 1 << bit)
        x = torch.stack([y[:, :, 0] + y[:, :, 1], y[:, :, 0] - y[:, :, 1]], 2).view(-1, 128)
    return (x / 128 ** 0.5).view(shape)


def _exact_codes(x):
    """What 64-bit rows stand for when they are held in 4 bits, by numpy's own rounding."""
    a = np.clip(x.cpu().numpy(), -4096.0, 4096.0)
    low = a.min(-1, keepdims=True)
    scale = ((a.max(-1, keepdims=True) - low) / 15).astype(np.float16).astype(np.float64)
    offset = (low - 64 * scale).astype(np.float16).astype(np.float64)
    with np.errstate(divide="ignore", invalid="ignore"):
        code = np.where(scale > 0, np.clip(np.rint((a - offset) / scale), 64, 79), 64)
    return torch.from_numpy((scale * code + offset).astype(np.float16).astype(np.float64)).cuda()


def _exact_rotary(c, s):
    n, kv = _lengths(c)
    qs, ks, vs, first = [], [], [], 0
    wide = c["cache"] != "int4"
    if wide:
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
    half, m = c["rot"] // 2, c["factor"]
    for b, (many, have) in enumerate(zip(n, kv)):
        pos = torch.arange(have - many, have, device="cuda")
        turn = torch.polar(torch.full((many, 1, half), m, dtype=torch.float64, device="cuda"),
                           (pos.double()[:, None] * s["freq"].double())[:, None])
        a, b_ = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if c["pairs"] == "neighbours" else \
            (slice(0, half), slice(half, 2 * half))

        def rotated(x):
            z = torch.complex(x[..., a].contiguous(), x[..., b_].contiguous()) * turn
            x = x.clone()
            x[..., a], x[..., b_] = z.real, z.imag
            return x

        q, k, v = (s[w][first:first + many].double() for w in "qkv")
        if c["turn"]:
            q, k, v = _butterflies(q), _butterflies(k), _butterflies(v)
        q, k = rotated(q), rotated(k)
        if c["turn"]:
            q, k = _butterflies(q), _butterflies(k)
        qs.append(q)
        if wide:
            if c["cache"] == "fp8":
                k = (k / s["k_scale"].double()[:, None]).clamp(-448, 448)
                v = (v / s["v_scale"].double()[:, None]).clamp(-448, 448)
            ids = s["table"][b].long()[pos // c["page"]]
            for h in range(c["hkv"]):
                kc[ids, h, pos % c["page"]] = k[:, h]
                vc[ids, h, :, pos % c["page"]] = v[:, h]
        else:
            ko, vo = _exact_cached(s, b, have)
            ko[have - many:], vo[have - many:] = _exact_codes(k), _exact_codes(v)
            ks.append(ko)
            vs.append(vo)
        first += many
    if wide:
        return {"q": torch.cat(qs), "k_cache": kc, "v_cache": vc}
    return {"q": torch.cat(qs), "k": torch.cat(ks), "v": torch.cat(vs)}


def _exact_probs(c, s):
    n, h, prompt = _token_lengths(c)
    out = torch.zeros(s["logits"].shape, dtype=torch.float64, device="cuda")
    history, drafts, row, at, draft = s["history"].long(), s["drafts"].long(), 0, 0, 0
    for b in range(c["b"]):
        t, repeats, presence, frequency = s["params"][b].double().tolist()
        told = history[at:at + prompt[b]]
        for j in range(n[b] + 1):
            made = torch.cat([history[at + prompt[b]:at + h[b]], drafts[draft:draft + j]])
            x = s["logits"][row].double()
            if s["bias"] is not None:
                ids, values, cu = s["bias"]
                mine = slice(int(cu[b]), int(cu[b + 1]))
                x[ids[mine].long()] += values[mine].double()
            seen = torch.unique(torch.cat([told, made]))
            y = x[seen]
            x[seen] = torch.where(y > 0, y / repeats, y * repeats)
            ids, times = torch.unique(made, return_counts=True)
            x[ids] -= frequency * times.double() + presence
            if s["mask"] is not None and int(s["mask_row"][row]) >= 0:
                words = s["mask"][int(s["mask_row"][row])].cpu().numpy().astype("<i4")
                bits = np.unpackbits(words.view(np.uint8), bitorder="little")[:c["vocab"]]
                x[torch.from_numpy(bits == 0).cuda()] = -math.inf
            if bool((x > -math.inf).any()):
                if t > 0:
                    out[row] = torch.softmax(x / t, 0)
                else:
                    out[row, int(torch.nonzero(x == x.max())[0, 0])] = 1.0
            row += 1
        at += h[b]
        draft += n[b]
    return {"p": out}

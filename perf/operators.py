"""The serving operators around the ternary products, as cases to be measured.

A decoder step with this library's products needs, between and after them: the
boundary of a block (its output's norm, gate, residual scale and residual, then
the next block's norm, with the rotations of the products on both sides), the
key/value cache in pages, the attention of a chunk of new tokens over it, and
the verification of drafted tokens.  `run` computes one call of one of them,
in elementary torch operations where `own` is false and by the library's entry
points where it is true.

Sizes: 5120 channels, 40 heads of 128 and batches up to 16 are the decoder
layer of this repository's benchmark; 8 key/value heads, chunks, vocabularies,
page sizes and lengths are generic.
"""

import math
import random

import torch

own = False

EPS = 1e-6


# ------------------------------------------------------------------- cases

def _attn(name, b, chunk, kv, hq, hkv, d, page, cache, window, ragged):
    return {"name": name, "op": "attention", "b": b, "chunk": chunk, "kv": kv, "hq": hq, "hkv": hkv, "d": d,
            "page": page, "cache": cache, "window": window, "ragged": ragged}


def _append(name, b, chunk, kv, hkv, d, page, cache, ragged):
    return {"name": name, "op": "append", "b": b, "chunk": chunk, "kv": kv, "hkv": hkv, "d": d, "page": page,
            "cache": cache, "ragged": ragged}


def _norm(name, rows, c, parts, stream, gate, rot_in, rot_out):
    return {"name": name, "op": "norm", "rows": rows, "c": c, "parts": parts, "stream": stream, "gate": gate,
            "rot_in": rot_in, "rot_out": rot_out}


def _verify(name, b, drafts, vocab, kind, one_hot):
    return {"name": name, "op": "verify", "b": b, "drafts": drafts, "vocab": vocab, "kind": kind, "one_hot": one_hot}


def listed():
    return [
        # one user's next token, a key/value head for each query head, small pages: latency
        _attn("attention-step-1", 1, 1, 1000, 40, 40, 128, 16, "bf16", 0, False),
        # a full decode batch at mixed lengths, shared heads
        _attn("attention-step-16", 16, 1, 8192, 40, 8, 128, 64, "bf16", 0, True),
        # few users with long contexts in an 8-bit cache
        _attn("attention-step-long-fp8", 4, 1, 65536, 40, 8, 128, 64, "fp8", 0, True),
        # a speculative step: a few drafted tokens a sequence
        _attn("attention-draft", 8, 9, 16384, 40, 8, 128, 32, "bf16", 0, True),
        # chunks of prompts over what is cached of them
        _attn("attention-chunk", 4, 2048, 8192, 40, 8, 128, 64, "bf16", 0, True),
        # a sliding window, odd lengths, 64-wide heads, an 8-bit cache in small pages
        _attn("attention-chunk-window-fp8", 2, 777, 6000, 16, 16, 64, 16, "fp8", 1000, False),
        # a decode batch's new keys and values
        _append("append-step-16", 16, 1, 256, 8, 128, 16, "bf16", True),
        # prompt chunks into an 8-bit cache
        _append("append-chunk-fp8", 4, 2048, 2500, 8, 128, 64, "fp8", True),
        # a block boundary of single-user decode: split product in, rotated operand out
        _norm("norm-step-1", 1, 5120, 4, "fp32", "none", True, True),
        # a block boundary of a prompt chunk, a gate for each token
        _norm("norm-chunk-2048", 2048, 5120, 1, "bf16", "token", False, True),
        # one user's drafted tokens, a small odd vocabulary
        _verify("verify-1", 1, 4, 32003, "fp32", False),
        # a batch of drafts over a large odd vocabulary
        _verify("verify-32", 32, 8, 131073, "fp32", False),
    ]


def _log(rng, lo, hi):
    """A whole number from lo to hi, even over its logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def _drawn(rng):
    op = rng.choice(["attention", "attention", "append", "norm", "verify"])
    cache, page = rng.choice(["bf16", "fp8"]), rng.choice([16, 32, 64, 128])
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 4, 8, 8, 10, 40])
    if op == "attention":
        group = rng.choice([1, 2, 4, 5, 8]) if hkv <= 8 else 1
        chunk = rng.choice([1, _log(rng, 1, 16), _log(rng, 1, 2048)])
        kv = max(chunk, _log(rng, 1, 65536 if chunk <= 16 else 8192))
        window = rng.choice([0, 0, _log(rng, 1, 4096)])
        c = _attn("", _log(rng, 1, 16), chunk, kv, hkv * group, hkv, d, page, cache, window, rng.random() < 0.6)
    elif op == "append":
        chunk = rng.choice([1, _log(rng, 1, 2048)])
        c = _append("", _log(rng, 1, 16), chunk, max(chunk, _log(rng, 1, 2500)), hkv, d, page, cache, rng.random() < 0.6)
    elif op == "norm":
        rows, parts, rot = _log(rng, 1, 2048), 1, rng.random() < 0.5
        if rows <= 16 and rot:
            parts = rng.choice([1, 2, 4, 8])
        c = _norm("", rows, 128 * _log(rng, 1, 40), parts, rng.choice(["bf16", "fp32"]),
                  rng.choice(["none", "channel", "token"]), rot, rng.random() < 0.6)
    else:
        c = _verify("", _log(rng, 1, 32), rng.randint(1, 8), _log(rng, 500, 131073), rng.choice(["fp32", "bf16"]),
                    rng.random() < 0.3)
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
        room = c["op"] in ("verify", "norm") or c["b"] * c["kv"] * c["hkv"] * c["d"] <= 1 << 28
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


def _draft_lengths(c):
    r = random.Random("%(b)d %(drafts)d %(vocab)d" % c)
    return [c["drafts"]] + [r.randint(0, c["drafts"]) for _ in range(c["b"] - 1)]


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


def _cache(shape, kind, g):
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.bfloat16)
    if kind == "fp8":
        # a head's scale puts its values in the middle of e4m3's range
        return (x * 8).to(torch.float8_e4m3fn)
    return x


def _cached(c, seed):
    n, kv = _lengths(c)
    g = _gen(seed)
    table, pages = _pages(c, kv, seed)
    s = {"op": c["op"], "n": n, "max_q": max(n), "max_kv": max(kv), "page": c["page"]}
    s["cu"], s["kv_len"], s["table"] = _ints(_offsets(n)), _ints(kv), _ints(table)
    s["k_cache"] = _cache((pages, c["hkv"], c["page"], c["d"]), c["cache"], g)
    s["v_cache"] = _cache((pages, c["hkv"], c["d"], c["page"]), c["cache"], g)
    s["k_scale"] = s["v_scale"] = None
    if c["cache"] == "fp8":
        s["k_scale"] = (0.1 + 0.05 * torch.rand(c["hkv"], generator=g, device="cuda"))
        s["v_scale"] = (0.1 + 0.05 * torch.rand(c["hkv"], generator=g, device="cuda"))
    return s, g


def _randn(shape, g, kind=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(kind)


def _hadamard(dtype):
    h = torch.ones(1, 1, dtype=dtype, device="cuda")
    while h.shape[0] < 128:
        h = torch.cat([torch.cat([h, h], 1), torch.cat([h, -h], 1)], 0)
    return h / math.sqrt(128.0)


def prepare(case, seed):
    c = case
    if c["op"] == "attention":
        s, g = _cached(c, seed)
        # the queries as a slice of a fused projection's output: a stride between tokens
        fused = _randn((sum(s["n"]), c["hq"] + 2 * c["hkv"], c["d"]), g, torch.bfloat16)
        s["q"] = fused[:, :c["hq"]]
        s["scale"], s["window"] = 1.5 / math.sqrt(c["d"]), c["window"]
        return s
    if c["op"] == "append":
        s, g = _cached(c, seed)
        fused = _randn((sum(s["n"]), 2 * c["hkv"], c["d"]), g, torch.bfloat16)
        s["k"], s["v"] = fused[:, :c["hkv"]], fused[:, c["hkv"]:]
        return s
    g = _gen(seed)
    if c["op"] == "norm":
        rows, ch, kind = c["rows"], c["c"], _KIND[c["stream"]]
        y = _randn((c["parts"], rows, ch), g, torch.float32 if c["parts"] > 1 or c["rot_in"] else torch.bfloat16)
        s = {"op": "norm", "y": y if c["parts"] > 1 else y[0], "parts": c["parts"], "resid": _randn((rows, ch), g, kind) * 3}
        s["w_post"] = (1 + 0.1 * _randn((ch,), g)).to(torch.bfloat16)
        s["w_pre"] = (1 + 0.1 * _randn((ch,), g)).to(torch.bfloat16)
        s["gate"], s["rows_per_gate"] = None, 0
        if c["gate"] == "channel":
            s["gate"], s["rows_per_gate"] = _randn((1, ch), g, torch.bfloat16), rows
        if c["gate"] == "token":
            s["gate"], s["rows_per_gate"] = _randn((rows, ch), g, torch.bfloat16), 1
        s["alpha"], s["rot_in"], s["rot_out"] = 0.7, c["rot_in"], c["rot_out"]
        s["hadamard"] = _hadamard(torch.float32)
        return s
    n = _draft_lengths(c)
    t, v, kind = sum(n), c["vocab"], _KIND[c["kind"]]
    logits = _randn((t + c["b"], v), g) * 2.5
    p = torch.softmax(logits, -1).to(kind)
    # target row of each drafted token, and a drafter that is near the target
    rows = [x for b, m in enumerate(n) for x in range(_offsets(n)[b] + b, _offsets(n)[b] + b + m)]
    at = torch.tensor(rows, dtype=torch.int64, device="cuda")
    q = torch.softmax(logits[at] + 0.5 * _randn((t, v), g), -1).to(kind)
    drafts = torch.argmax(q.float() / torch.empty((t, v), device="cuda").exponential_(generator=g), -1).to(torch.int32) \
        if t else torch.zeros(0, dtype=torch.int32, device="cuda")
    return {"op": "verify", "p": p, "q": None if c["one_hot"] else q, "drafts": drafts, "cu": _ints(_offsets(n)),
            "max_draft": max(n), "u": torch.rand(t, generator=g, device="cuda"),
            "u_next": torch.rand(c["b"], generator=g, device="cuda")}


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


def _plain_attention(s):
    tokens, hq, d = s["q"].shape
    hkv = s["k_cache"].shape[1]
    group, nb, nq, nk = hq // hkv, s["kv_len"].shape[0], s["max_q"], s["max_kv"]
    page, slot, live = _positions(s, nk)
    k = s["k_cache"][page, :, slot].float()                                # [B, L, Hkv, D]
    v = s["v_cache"][page, :, :, slot].float() * live[:, :, None, None]
    if s["k_scale"] is not None:
        k, v = k * s["k_scale"][None, None, :, None], v * s["v_scale"][None, None, :, None]
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


def _plain_append(s):
    b, _, pos = _owners(s)
    page, slot = s["table"].long()[b, pos // s["page"]], pos % s["page"]
    k, v, kind = s["k"].float(), s["v"].float(), s["k_cache"].dtype
    if s["k_scale"] is not None:
        k = (k / s["k_scale"][None, :, None]).clamp(-448.0, 448.0)
        v = (v / s["v_scale"][None, :, None]).clamp(-448.0, 448.0)
    as_bits = torch.uint8 if kind == torch.float8_e4m3fn else torch.int16
    s["k_cache"].view(as_bits)[page, :, slot] = k.to(kind).view(as_bits)
    s["v_cache"].view(as_bits)[page, :, :, slot] = v.to(kind).view(as_bits)
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_norm(s):
    u = s["y"].float()
    if s["parts"] > 1:
        u = u.sum(0)
    if s["rot_in"]:
        u = (u.view(-1, 128) @ s["hadamard"]).view(u.shape)
    u = u * torch.rsqrt(u.square().mean(-1, keepdim=True) + EPS) * s["w_post"].float()
    if s["gate"] is not None:
        u = u * s["gate"].float()
    h = s["resid"].float() + s["alpha"] * u
    z = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["w_pre"].float()
    if s["rot_out"]:
        z = (z.view(-1, 128) @ s["hadamard"]).view(z.shape)
    return {"h": h.to(s["resid"].dtype), "z": z.to(torch.bfloat16)}


def _plain_verify(s):
    p, q, cu = s["p"], s["q"], s["cu"].long()
    nb, v, t = cu.shape[0] - 1, p.shape[1], s["max_draft"]
    n = cu[1:] - cu[:-1]
    seq = torch.arange(nb, device="cuda")
    j = torch.arange(t, device="cuda")
    live = j[None] < n[:, None]
    at = torch.where(live, cu[:-1, None] + j[None], 0)
    d = s["drafts"].long()[at]
    pd = p[at + seq[:, None], d].double()
    qd = torch.ones_like(pd) if q is None else q[at, d].double()
    kept = (s["u"].double()[at] * qd < pd) & live
    count = torch.cumprod(kept.long(), 1).sum(1)
    row = p[cu[:-1] + seq + count].double()
    last = torch.where(count < n, cu[:-1] + count, 0)
    if q is None:
        less = torch.zeros_like(row)
        less.scatter_(1, s["drafts"].long()[last][:, None], math.inf)
    else:
        less = q[last].double()
    rest = (row - less).clamp(min=0.0)
    rest = torch.where((count < n)[:, None], rest, row)
    rest = torch.where(rest.sum(1, keepdim=True) > 0, rest, row)
    total = torch.cumsum(rest, 1)
    token = (total <= s["u_next"].double()[:, None] * total[:, -1:]).sum(1)
    highest = v - 1 - torch.argmax((rest.flip(1) > 0).long(), 1)
    token = torch.minimum(token, highest)
    tokens = torch.full((nb, t + 1), -1, dtype=torch.int64, device="cuda")
    tokens[:, :t] = torch.where(j[None] < count[:, None], d, -1)
    tokens[seq, count] = token
    return {"accepted": count.to(torch.int32), "tokens": tokens.to(torch.int32)}


# -------------------------------------------------------------------- run

def run(state):
    s = state
    if not own:
        return {"attention": _plain_attention, "append": _plain_append, "norm": _plain_norm,
                "verify": _plain_verify}[s["op"]](s)
    from ternary_weights_hadamard_amd import tb
    if s["op"] == "attention":
        out, lse = tb.tb_paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["cu"], s["kv_len"],
                                         s["max_q"], s["max_kv"], scale=s["scale"], window=s["window"],
                                         k_scale=s["k_scale"], v_scale=s["v_scale"], with_lse=True)
        return {"out": out, "lse": lse}
    if s["op"] == "append":
        tb.tb_paged_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["cu"], s["kv_len"], s["max_q"],
                           k_scale=s["k_scale"], v_scale=s["v_scale"])
        return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if s["op"] == "norm":
        h, z = tb.tb_block_norm(s["y"], s["resid"], w_post=s["w_post"], w_pre=s["w_pre"], gate=s["gate"],
                                rows_per_gate=s["rows_per_gate"], alpha=s["alpha"], eps=EPS, y_parts=s["parts"],
                                rotate_in=s["rot_in"], rotate_out=s["rot_out"])
        return {"h": h, "z": z}
    accepted, tokens = tb.tb_verify_draft(s["p"], s["q"], s["drafts"], s["u"], s["u_next"], s["cu"], s["max_draft"])
    return {"accepted": accepted, "tokens": tokens}


def work(case):
    c = case
    if c["op"] in ("attention", "append"):
        n, kv = _lengths(c)
        size = 1 if c["cache"] == "fp8" else 2
        row = c["hkv"] * c["d"]
        if c["op"] == "append":
            return {"bytes": 2.0 * sum(n) * row * (2 + size), "flops": 0.0}
        keys, pairs = 0, 0
        for m, have in zip(n, kv):
            w = c["window"] or have
            keys += min(have, w + m - 1)
            # the token at position x sees min(x + 1, w) keys
            first = have - m
            short = max(0, min(m, w - first))
            pairs += short * (first + 1) + short * (short - 1) // 2 + (m - short) * w
        return {"bytes": 2.0 * keys * row * size + sum(n) * c["hq"] * (4.0 * c["d"] + 4),
                "flops": 4.0 * c["d"] * c["hq"] * pairs}
    if c["op"] == "norm":
        size = 2 if c["stream"] == "bf16" else 4
        y = c["parts"] * (4 if c["parts"] > 1 or c["rot_in"] else 2)
        gate = {"none": 0, "channel": 2.0 / c["rows"], "token": 2}[c["gate"]]
        return {"bytes": c["rows"] * c["c"] * (y + 2 * size + 2 + gate) + 4.0 * c["c"],
                "flops": c["rows"] * c["c"] * (12.0 + 14 * (c["rot_in"] + c["rot_out"]))}
    n = _draft_lengths(c)
    size = 2 if c["kind"] == "bf16" else 4
    # one row of the target's a sequence, and one of the drafter's for most
    return {"bytes": c["b"] * c["vocab"] * size * (1.0 if c["one_hot"] else 2.0) + 12.0 * sum(n) + 4.0 * c["b"] * (c["drafts"] + 3),
            "flops": 3.0 * c["b"] * c["vocab"]}


# ------------------------------------------------------------------ exact

def exact(case, seed):
    """The definitions, sequence by sequence, in 64 bits."""
    c, s = case, prepare(case, seed)
    if c["op"] == "attention":
        return _exact_attention(c, s)
    if c["op"] == "append":
        return _exact_append(c, s)
    if c["op"] == "norm":
        return _exact_norm(c, s)
    return _exact_verify(c, s)


def _exact_attention(c, s):
    n, kv = _lengths(c)
    group, outs, lses, first = c["hq"] // c["hkv"], [], [], 0
    for b, (m, have) in enumerate(zip(n, kv)):
        ids = s["table"][b, :-(-have // c["page"])].long()
        k = s["k_cache"][ids].double().transpose(1, 2).reshape(-1, c["hkv"], c["d"])[:have]
        v = s["v_cache"][ids].double().permute(0, 3, 1, 2).reshape(-1, c["hkv"], c["d"])[:have]
        pos = torch.arange(have - m, have, device="cuda")[:, None]
        key = torch.arange(have, device="cuda")[None]
        hide = (key > pos) | ((key <= pos - c["window"]) if c["window"] else torch.zeros_like(key, dtype=torch.bool))
        out = torch.empty((m, c["hq"], c["d"]), dtype=torch.float64, device="cuda")
        lse = torch.empty((m, c["hq"]), dtype=torch.float64, device="cuda")
        for h in range(c["hq"]):
            kh, vh = k[:, h // group], v[:, h // group]
            if s["k_scale"] is not None:
                kh, vh = kh * s["k_scale"][h // group].double(), vh * s["v_scale"][h // group].double()
            x = (s["q"][first:first + m, h].double() @ kh.T.contiguous()) * s["scale"]
            x[hide] = -math.inf
            lse[:, h] = torch.logsumexp(x, 1)
            out[:, h] = torch.exp(x - lse[:, h, None]) @ vh
        outs.append(out)
        lses.append(lse)
        first += m
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}


def _exact_append(c, s):
    n, kv = _lengths(c)
    kc, vc, first = s["k_cache"].double(), s["v_cache"].double(), 0
    for b, (m, have) in enumerate(zip(n, kv)):
        k, v = s["k"][first:first + m].double(), s["v"][first:first + m].double()
        if s["k_scale"] is not None:
            k = (k / s["k_scale"].double()[:, None]).clamp(-448, 448)
            v = (v / s["v_scale"].double()[:, None]).clamp(-448, 448)
        pos = torch.arange(have - m, have, device="cuda")
        ids = s["table"][b].long()[pos // c["page"]]
        for h in range(c["hkv"]):
            kc[ids, h, pos % c["page"]] = k[:, h]
            vc[ids, h, :, pos % c["page"]] = v[:, h]
        first += m
    return {"k_cache": kc, "v_cache": vc}


def _exact_norm(c, s):
    u = s["y"].double()
    u = sum(u[i] for i in range(c["parts"])) if c["parts"] > 1 else u
    had = _hadamard(torch.float64)

    def turned(x):
        return torch.cat([x[:, i:i + 128] @ had for i in range(0, c["c"], 128)], 1)

    def normed(x, w):
        return x / torch.sqrt((x * x).sum(1, keepdim=True) / c["c"] + EPS) * w.double()

    a = normed(turned(u) if c["rot_in"] else u, s["w_post"])
    if s["gate"] is not None:
        a = s["gate"].double() * a
    h = s["resid"].double() + s["alpha"] * a
    z = normed(h, s["w_pre"])
    return {"h": h, "z": turned(z) if c["rot_out"] else z}


def _exact_verify(c, s):
    n, first, counts = _draft_lengths(c), 0, []
    tokens = torch.full((c["b"], s["max_draft"] + 1), -1, dtype=torch.int32)
    drafts, u = s["drafts"].tolist(), s["u"].tolist()
    for b, m in enumerate(n):
        count = 0
        while count < m:
            d = drafts[first + count]
            ratio = 1.0 if s["q"] is None else float(s["q"][first + count, d])
            if not u[first + count] * ratio < float(s["p"][first + b + count, d]):
                break
            tokens[b, count] = d
            count += 1
        w = s["p"][first + b + count].double().cpu()
        if count < m:
            if s["q"] is None:
                r = w.clone()
                r[drafts[first + count]] = 0
            else:
                r = (w - s["q"][first + count].double().cpu()).clamp(min=0)
            w = r if float(r.sum()) > 0 else w
        edge = torch.cumsum(w, 0)
        token = int((edge <= float(s["u_next"][b]) * float(edge[-1])).sum())
        tokens[b, count] = min(token, int(torch.nonzero(w)[-1]))
        counts.append(count)
        first += m
    return {"accepted": torch.tensor(counts, dtype=torch.int32), "tokens": tokens}

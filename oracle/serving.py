"""The serving operators around the products, from their formulas (include/tb.h),
in float64 and one row at a time: the boundary of a block, the paged cache, the
attention over it, the verification of drafted tokens.  Pinned by
tests/test_oracle_serving.py against worked cases.
"""

import numpy as np

from . import hadamard


def block_norm(y, resid, w_post, w_pre, gate, rows_per_gate, alpha, eps, rotate_in, rotate_out):
    """(h, z) of float64 arrays: y [parts, rows, C] or None, the others [rows, C],
    [C] or [gates, C], or None."""
    if y is None:
        h = resid.copy()
    else:
        u = y.sum(0)
        if rotate_in:
            u = hadamard.fwht_dense(u)
        if w_post is not None:
            u = u / np.sqrt((u * u).mean(1, keepdims=True) + eps) * w_post
        if gate is not None:
            u = u * gate[np.arange(u.shape[0]) // rows_per_gate]
        h = alpha * u + (0.0 if resid is None else resid)
    z = None
    if w_pre is not None:
        z = h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * w_pre
        if rotate_out:
            z = hadamard.fwht_dense(z)
    return h, z


def paged_rows(cu, kv_len, b):
    """(row, position) of sequence b's tokens."""
    lo, hi = int(cu[b]), int(cu[b + 1])
    return [(r, int(kv_len[b]) - (hi - lo) + r - lo) for r in range(lo, hi)]


def paged_slot(table, page, n_pages, b, pos):
    """(page id, slot) of a position, or None where there is none."""
    if pos < 0 or pos // page >= table.shape[1]:
        return None
    i = int(table[b, pos // page])
    return (i, pos % page) if 0 <= i < n_pages else None


def paged_gather(k_cache, v_cache, table, page, b, positions):
    """Keys and values [len, heads, d] of positions that exist, and those positions."""
    got, ks, vs = [], [], []
    for x in positions:
        at = paged_slot(table, page, k_cache.shape[0], b, x)
        if at is not None:
            got.append(x)
            ks.append(k_cache[at[0], :, at[1]])
            vs.append(v_cache[at[0], :, :, at[1]])
    heads, d = k_cache.shape[1], k_cache.shape[3]
    return (np.array(ks).reshape(-1, heads, d), np.array(vs).reshape(-1, heads, d), np.array(got, dtype=np.int64))


def paged_attention(q, k_cache, v_cache, table, cu, kv_len, scale, window):
    """out [tokens, heads_q, d], lse, and what error bounds are made of: the
    weighted mean magnitude of the values (like out) and the largest sum
    |q_i k_i| * |scale| of a seen score (like lse).  Caches are float64
    [pages, heads, page, d] and [pages, heads, d, page]."""
    tokens, hq, d = q.shape
    hkv, page = k_cache.shape[1], k_cache.shape[2]
    out, mean = np.zeros((tokens, hq, d)), np.zeros((tokens, hq, d))
    lse, size = np.full((tokens, hq), -np.inf), np.zeros((tokens, hq))
    for b in range(len(kv_len)):
        rows = paged_rows(cu, kv_len, b)
        if not rows:
            continue
        low = max(0, rows[0][1] - window + 1) if window else 0
        k, v, at = paged_gather(k_cache, v_cache, table, page, b, range(low, max(0, rows[-1][1] + 1)))
        for r, pos in rows:
            see = (at <= pos) & ((at > pos - window) if window else True)
            if not see.any():
                continue
            for h in range(hq):
                kh, vh = k[see, h // (hq // hkv)], v[see, h // (hq // hkv)]
                s = kh @ q[r, h] * scale
                size[r, h] = np.max(np.abs(kh) @ np.abs(q[r, h])) * abs(scale)
                top = s.max()
                w = np.exp(s - top)
                lse[r, h] = top + np.log(w.sum())
                out[r, h] = w @ vh / w.sum()
                mean[r, h] = w @ np.abs(vh) / w.sum()
    return out, lse, mean, size


def verify_draft(p, q, drafts, u, u_next, cu, max_draft):
    """(accepted [B], tokens [B, max_draft + 1]) of float64 probabilities; q may be None."""
    nb, vocab = len(u_next), p.shape[1]
    accepted, tokens = np.zeros(nb, np.int32), np.full((nb, max_draft + 1), -1, np.int32)

    def weights(x):
        return np.where((x > 0) & (x < np.inf), x, 0.0)

    for b in range(nb):
        lo, n = int(cu[b]), int(cu[b + 1]) - int(cu[b])
        m = 0
        while m < n:
            d = int(drafts[lo + m])
            if not 0 <= d < vocab:
                break
            if not u[lo + m] * (1.0 if q is None else q[lo + m, d]) < p[lo + b + m, d]:
                break
            tokens[b, m] = d
            m += 1
        w = weights(p[lo + b + m])
        if m < n:
            if q is None:
                rest = w.copy()
                if 0 <= drafts[lo + m] < vocab:
                    rest[drafts[lo + m]] = 0.0
            else:
                with np.errstate(invalid="ignore"):
                    rest = weights(p[lo + b + m] - q[lo + m])
            if rest.sum() > 0:
                w = rest
        accepted[b] = m
        if w.sum() > 0:
            edge = np.cumsum(w)
            past = np.nonzero((edge > u_next[b] * edge[-1]) & (w > 0))[0]
            tokens[b, m] = past[0] if len(past) else np.nonzero(w)[0][-1]
    return accepted, tokens

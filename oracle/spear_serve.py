"""Float64 oracle of the serving operators: the paged key/value cache, attention
over it, and the verification of drafted tokens.  Plain loops over sequences,
heads and tokens; nothing is shared with the HIP path."""
import numpy as np


def quantise_kv(x):
    """8-bit form of fp16 rows [..., head_dim]: (codes int8, scales fp32 [...]).

    s = max|x| / 127 and code = rint(x / s), both divisions in float32 (so the
    codes are the definition's), ties to even, 0 where s = 0 or not finite."""
    x = np.asarray(x, dtype=np.float32)
    with np.errstate(all="ignore"):
        s = (np.abs(x).max(-1) / np.float32(127)).astype(np.float32)
        c = np.rint(x / s[..., None])
    c = np.where((s > 0)[..., None] & np.isfinite(c), c, 0)
    return np.clip(c, -127, 127).astype(np.int8), s


def cached(cache, scale, table_row, n):
    """The first n cached tokens of a sequence in float64 [n, heads, head_dim]."""
    page = cache.shape[2]
    rows = []
    for i in range(n):
        p, o = int(table_row[i // page]), i % page
        x = cache[p, :, o].astype(np.float64)
        if scale is not None:
            x = x * scale[p, :, o].astype(np.float64)[:, None]
        rows.append(x)
    return np.stack(rows) if rows else np.zeros((0, cache.shape[1], cache.shape[3]))


def paged_attention(q, k_cache, v_cache, table, cu_q, kv_lens, scale, k_scale=None, v_scale=None):
    """(out, spread, reach): out float64 [total_q, q_heads, head_dim]; what bounds the
    error of an implementation: spread, the weighted mean of |v| per element, and
    reach, the largest sum of |q_d k_d| over visible keys, times scale, per row and head."""
    total, heads, dim = q.shape
    group = heads // k_cache.shape[1]
    out = np.zeros((total, heads, dim))
    spread, reach = np.zeros_like(out), np.zeros((total, heads))
    for b in range(len(kv_lens)):
        n, length = int(cu_q[b + 1] - cu_q[b]), int(kv_lens[b])
        if n == 0:
            continue
        k = cached(k_cache, k_scale, table[b], length)
        v = cached(v_cache, v_scale, table[b], length)
        for i in range(n):
            seen = min(length, length - n + i + 1)
            if seen <= 0:
                continue
            for h in range(heads):
                x = q[cu_q[b] + i, h].astype(np.float64)
                kk, vv = k[:seen, h // group], v[:seen, h // group]
                z = kk @ x * scale
                if np.all(np.isneginf(z)):
                    continue
                p = np.exp(z - z.max())
                p /= p.sum()
                row = cu_q[b] + i
                out[row, h] = p @ vv
                spread[row, h] = p @ np.abs(vv)
                reach[row, h] = (np.abs(kk) @ np.abs(x)).max() * scale
    return out, spread, reach


def verify_draft(target, draft, drafted, u, noise, num_drafts=None):
    """(accepted [B], tokens [B, K + 1]) by the definition; decisions in float32,
    as the definition states, one element at a time."""
    B, K1, V = target.shape
    K = K1 - 1
    f = np.float32
    accepted = np.zeros(B, dtype=np.int32)
    tokens = np.full((B, K1), -1, dtype=np.int32)
    for b in range(B):
        n = K if num_drafts is None else int(min(max(num_drafts[b], 0), K))
        a = 0
        while a < n:
            x = int(drafted[b, a])
            if not 0 <= x < V:
                break
            q = f(1) if draft is None else f(draft[b, a, x])
            if not f(u[b, a]) * q < f(target[b, a, x]):
                break
            tokens[b, a] = x
            a += 1
        accepted[b] = a
        p = target[b, a].astype(np.float32)
        w = p
        if a < n:
            if draft is None:
                q = np.zeros(V, dtype=np.float32)
                if 0 <= drafted[b, a] < V:
                    q[drafted[b, a]] = 1
            else:
                q = draft[b, a].astype(np.float32)
            w = p - q
        for weights in ((w, p) if a < n else (p,)):
            best, token = None, -1
            with np.errstate(all="ignore"):
                score = weights / noise[b].astype(np.float32)
            for j in np.nonzero((weights > 0) & (score >= 0))[0]:
                if best is None or score[j] > best:
                    best, token = score[j], int(j)
            if token >= 0:
                break
        tokens[b, a] = token
    return accepted, tokens

"""Oracle of what a serving step does around the layers and the cache: its pages,
block tables and slots, the adapters of its requests, and the draw of its next
tokens, in 64 bits.  Plain loops over sequences and tokens; nothing is shared with the
HIP path."""
import numpy as np


def kv_plan(lens, new_tokens, held, table, free_pages, free_count, rows, page):
    """(cu_q, kv_lens, slots, positions, sequence, held, free_count, table, free_pages)
    after the step, by the definition: one sequence and one page at a time."""
    B, max_pages = table.shape
    table, free_pages = table.copy(), free_pages.copy()
    stack = [int(x) for x in free_pages[:min(max(int(free_count), 0), len(free_pages))]]
    old = len(stack)
    want, valid = [], []
    for b in range(B):
        want.append(-(-(int(lens[b]) + int(new_tokens[b])) // page))
        valid.append(lens[b] >= 0 and new_tokens[b] >= 0 and 0 <= held[b] <= max_pages and want[b] <= max_pages
                     and int(held[b]) * page >= lens[b])
    now = [int(h) for h in held]
    for b in range(B):
        if valid[b]:
            stack += [int(x) for x in table[b, want[b]:now[b]]]
            now[b] = min(now[b], max(want[b], 0))
    laid = list(stack)
    n, full = [0] * B, False
    for b in range(B):
        if not valid[b] or full:
            continue
        need = want[b] - now[b]
        if need > len(stack) or sum(n) + int(new_tokens[b]) > rows:
            full = True
            continue
        for e in range(now[b], want[b]):
            table[b, e] = stack.pop()
        now[b], n[b] = want[b], int(new_tokens[b])
    stack = stack[:len(free_pages)]
    for i in range(old, len(stack)):
        free_pages[i] = laid[i]
    cu = np.concatenate([[0], np.cumsum(n)]).astype(np.int32)
    slots = np.full(rows, -1, np.int64)
    positions, sequence = np.full(rows, -1, np.int32), np.full(rows, -1, np.int32)
    for b in range(B):
        for i in range(n[b]):
            r, p = int(cu[b]) + i, int(lens[b]) + i
            positions[r], sequence[r] = p, b
            slots[r] = int(table[b, p // page]) * page + p % page
    kv_lens = (np.asarray(lens, np.int64) + n).astype(np.int32)
    return (cu, kv_lens, slots, positions, sequence, np.asarray(now, np.int32), np.asarray([len(stack)], np.int32), table,
            free_pages)


def adapter_add(Y, X, A, B, cu, adapter, scale=None):
    """(out, slack) float64 [rows, N]: Y + scale[a] (X A[a]^T) B[a]^T for the rows of
    sequences with an adapter; slack bounds the error of an implementation that holds
    sums in fp32 and H = X A^T to 2^-22 of its row's largest, before its last rounding:
    K roundings of 2^-24 of each sum of H, 2 rank + 4 of the second product's."""
    out = Y.astype(np.float64)
    slack = np.zeros_like(out)
    K, rank = X.shape[1], A.shape[1]
    for b, a in enumerate(adapter):
        if not 0 <= a < len(A):
            continue
        at = slice(int(cu[b]), int(cu[b + 1]))
        x, wa, wb = X[at].astype(np.float64), A[a].astype(np.float64), B[a].astype(np.float64)
        s = 1.0 if scale is None else float(scale[a])
        h = x @ wa.T
        out[at] += s * (h @ wb.T)
        h_err = K * 2.0 ** -24 * (np.abs(x) @ np.abs(wa).T)
        if h.size:
            h_err += 2.0 ** -22 * np.abs(h).max(1, keepdims=True)
        slack[at] = abs(s) * (h_err @ np.abs(wb).T + (2 * rank + 4) * 2.0 ** -24 * (np.abs(h) @ np.abs(wb).T))
    return out, slack


def kept_tokens(logits, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, nudge=0.0):
    """(tokens, weights) that the rules leave of one row, in falling order; weights in
    64 bits relative to the largest.  `nudge`: relative change of top-p's mass, to ask
    how near its cut is to the next."""
    l = np.asarray(logits, np.float64)
    l = np.where(np.isnan(l), -np.inf, l)
    order = np.argsort(-l, kind="stable")
    order = order[l[order] > -np.inf]
    if not len(order) or not temperature > 0 or top_k == 1 or top_p <= 0:
        return order[:1], np.ones(min(len(order), 1))
    z = l[order]
    with np.errstate(all="ignore"):
        w = np.exp((z - z[0]) / float(temperature))
    w = np.where(z == z[0], 1.0, w)                     # (infinite ones too)
    w = np.where(w >= 2.0 ** -126, w, 0.0)
    n = len(w) if top_k <= 0 else min(top_k, len(w))
    n = min(n, int((w > 0).sum()))
    if top_p < 1:
        target = float(top_p) * w[:n].sum() * (1 + nudge)
        n = max(1, int((np.concatenate([[0.0], np.cumsum(w[:n])[:-1]]) < target).sum()))
    if min_p > 0:
        n = min(n, int((w[:n] >= min(float(min_p), 1.0)).sum()))
    return order[:n], w[:n]


def sample(logits, noise, *rules, nudge=0.0):
    """(token, scores, probabilities) of one row: the race in float32 as the definition
    states; scores by token (-1: not drawn), None without noise."""
    at, w = kept_tokens(logits, *rules, nudge=nudge)
    probs = np.zeros(len(logits))
    if not len(at):
        return -1, None, probs
    probs[at] = w / w.sum()
    if len(at) == 1 and noise is None:
        return int(at[0]), None, probs
    if noise is None:
        return None, None, probs
    scores = np.full(len(logits), -1.0, np.float32)
    with np.errstate(all="ignore"):
        s = w.astype(np.float32) / noise[at].astype(np.float32)
    scores[at] = np.where((s >= 0) & (w > 0), s, np.float32(-1))
    best = scores.max()
    return (int(np.argmax(scores)) if best >= 0 else -1), scores, probs

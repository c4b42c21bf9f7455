"""Workloads of what a serving step does around the W4 layers and the paged
cache: its pages, block tables and slots planned on the GPU; the low-rank
adapters of its requests added beside a shared projection; the next tokens
sampled from the logits with temperature, top-k, top-p and min-p.

Each case is run either in its plain form (elementary torch operations) or,
with `own` set, by the calls a user makes of the framework.
"""
import math
import random

import torch

own = False

DEVICE = "cuda"


# --------------------------------------------------------------------- cases

def listed():
    return [
        # A lightly loaded server's two requests with the usual settings: latency counts.
        dict(name="sample_small", op="sample", batch=2, vocab=32000, logits="fp16", rule="all", masked=0.0, draw=True,
             probs=False),
        # A full decode batch over a large vocabulary, every request with settings of its own.
        dict(name="sample_batch", op="sample", batch=64, vocab=128001, logits="fp16", rule="mixed", masked=0.0,
             draw=True, probs=False),
        # Temperature alone, fp32 logits; every token may be drawn.
        dict(name="sample_temperature", op="sample", batch=24, vocab=50257, logits="fp32", rule="temperature",
             masked=0.0, draw=True, probs=False),
        # The target's distribution at each position of drafted tokens, as the verification reads it.
        dict(name="sample_target", op="sample", batch=144, vocab=32000, logits="fp16", rule="top_p", masked=0.0,
             draw=False, probs=True),
        # Drafting under a grammar that forbids half of the vocabulary: tokens and their distribution.
        dict(name="sample_draft", op="sample", batch=16, vocab=100002, logits="fp16", rule="mixed", masked=0.5,
             draw=True, probs=True),
        # One token more for each of a batch's sequences.
        dict(name="plan_decode", op="plan", batch=96, page=16, max_len=8192, new="decode", chunk=0, short=False),
        # A large batch in which requests end, start and go back after refused drafts.
        dict(name="plan_mixed", op="plan", batch=1500, page=16, max_len=4096, new="mixed", chunk=301, short=False),
        # Long prompts' chunks, more of them than there are pages for.
        dict(name="plan_prompts", op="plan", batch=41, page=32, max_len=16384, new="prompts", chunk=4096, short=True),
        # One request with an adapter, one projection.
        dict(name="adapter_one", op="adapter", batch=1, rows=1, adapters=1, rank=16, shapes="4096x4096", bare=0.0),
        # A decode step's requests, each with one of 24 adapters or none, in the four adapted projections of a layer.
        dict(name="adapter_decode", op="adapter", batch=64, rows=64, adapters=24, rank=16,
             shapes="2048x2048,2048x2048,2048x8192,8192x2048", bare=0.1),
        # A prompt's chunk in one batch with the decode steps of 40 others, in a wide projection.
        dict(name="adapter_mixed", op="adapter", batch=41, rows=740, adapters=12, rank=32, shapes="14336x4096", bare=0.1),
        # Chunks of a few long prompts.
        dict(name="adapter_chunk", op="adapter", batch=5, rows=2048, adapters=4, rank=64, shapes="4096x14336", bare=0.0),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        c = _draw_any(rng)
        if _cost(c) <= most:
            return c


def _draw_any(rng):
    op = rng.choice(["sample", "sample", "plan", "adapter", "adapter"])
    if op == "sample":
        token = rng.random() < 0.7
        return dict(op=op, batch=_log_int(rng, 1, 256), vocab=_log_int(rng, 1000, 131071),
                    logits=rng.choice(["fp16", "fp16", "fp32"]),
                    rule=rng.choice(["all", "mixed", "temperature", "top_k", "top_p", "min_p"]),
                    masked=rng.choice([0.0, 0.0, 0.3, 0.95]), draw=token, probs=not token or rng.random() < 0.3)
    if op == "plan":
        new = rng.choice(["decode", "mixed", "prompts"])
        batch = _log_int(rng, 1, 100 if new == "prompts" else 4000)
        return dict(op=op, batch=batch, page=rng.choice([16, 32, 64]), max_len=_log_int(rng, 500, 20000), new=new,
                    chunk=0 if new == "decode" else _log_int(rng, 17, 5000 if batch < 100 else 400),
                    short=rng.random() < 0.4)
    rows = _log_int(rng, 1, 2048)
    K, N = (8 * _log_int(rng, 64, 1800) for _ in range(2))
    return dict(op=op, batch=rows if rows < 200 and rng.random() < 0.5 else rng.randint(1, min(rows, 48)), rows=rows,
                adapters=_log_int(rng, 1, 32), rank=rng.choice([8, 16, 32, 64, 128]),
                shapes="%dx%d" % (K, N + (rng.randint(1, 7) if rng.random() < 0.3 else 0)), bare=rng.choice([0.0, 0.2]))


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def _shapes(case):
    return [tuple(int(n) for n in s.split("x")) for s in case["shapes"].split(",")]


def _settings(case, r):
    """(temperature, top_k, top_p, min_p) of one request; 0, 0, 1 and 0 leave a rule out (greedy for the temperature)."""
    rule = case["rule"] if case["rule"] != "mixed" else r.choice(["all", "temperature", "top_k", "top_p", "min_p", "greedy"])
    t = 0.0 if rule == "greedy" else round(r.uniform(0.5, 1.3), 3)
    return (t, r.choice([20, 50, 200]) if rule in ("all", "top_k") else 0,
            round(r.uniform(0.7, 0.98), 3) if rule in ("all", "top_p") else 1.0,
            round(r.uniform(0.01, 0.1), 3) if rule in ("all", "min_p") else 0.0)


def _batch_settings(case):
    r = random.Random(case["batch"] * 7 + case["vocab"])
    return [_settings(case, r) for _ in range(case["batch"])]


def _request(case, r):
    """(cached tokens, new tokens, pages held) of one sequence."""
    page, n, new, kind = case["page"], _log_int(r, 1, case["max_len"]), 1, r.random()
    if case["new"] == "prompts":
        return (n, r.randint(1, case["chunk"]), -(-n // page)) if kind > 0.3 else (0, r.randint(1, case["chunk"]), 0)
    if case["new"] == "mixed" and kind < 0.05:
        return 0, _log_int(r, 1, case["chunk"]), 0              # it begins
    if case["new"] == "mixed" and kind < 0.1:
        return n, 0, -(-n // page)                              # it waits
    if case["new"] == "mixed" and kind > 0.95:
        return 0, 0, -(-n // page)                              # it has ended
    refused = case["new"] == "mixed" and kind > 0.8             # it went back after refused drafts
    return n, new, -(-n // page) + refused


def _requests(case):
    """Every sequence's _request(), and the pages that are free."""
    r = random.Random(case["batch"] * 31 + case["max_len"])
    got = [_request(case, r) for _ in range(case["batch"])]
    need = sum(max(0, -(-(n + new) // case["page"]) - held) for n, new, held in got)
    return got, max(1, need * 2 // 3) if case["short"] else need + 37


def _rows_of(case):
    """New rows of each sequence in an adapter case: single tokens, and the rest in the first sequences."""
    batch, rows = case["batch"], case["rows"]
    long = max(1, batch // 16) if rows > batch and batch > 8 else batch
    r = random.Random(case["rows"] * 13 + batch)
    spare, cuts = rows - batch, sorted(r.randint(0, rows - batch) for _ in range(long - 1))
    parts = [b - a for a, b in zip([0] + cuts, cuts + [spare])]
    return [1 + (parts[b] if b < long else 0) for b in range(batch)]


def _adapters_of(case):
    r = random.Random(case["rows"] * 17 + case["adapters"])
    return [-1 if r.random() < case["bare"] else r.randrange(case["adapters"]) for _ in range(case["batch"])]


def work(case):
    if case["op"] == "sample":
        b, v = case["batch"], case["vocab"]
        read = b * v * (2.0 if case["logits"] == "fp16" else 4.0)
        if case["draw"]:    # the noise of tokens that may be drawn: what top-k leaves, or all where there is no rule
            for t, k, p, m in _batch_settings(case):
                read += 4.0 * (0 if t == 0 else min(k, v) if k else 0 if p < 1 or m > 0 else v)
        return {"bytes": read + (4.0 * b * v if case["probs"] else 0) + 20.0 * b, "flops": 4.0 * b * v}
    if case["op"] == "plan":
        got, free = _requests(case)
        rows = sum(new for _, new, _ in got)
        pages = sum(max(0, -(-(n + new) // case["page"]) - held) for n, new, held in got)
        return {"bytes": 24.0 * len(got) + 16.0 * rows + 8.0 * min(pages, free), "flops": 8.0 * (len(got) + rows)}
    lens, which = _rows_of(case), _adapters_of(case)
    rows = sum(n for n, a in zip(lens, which) if a >= 0)
    used = len({a for a in which if a >= 0})
    nbytes = flops = 1.0
    for K, N in _shapes(case):
        nbytes += 2.0 * (used * case["rank"] * (K + N) + rows * (K + 2 * N))
        flops += 2.0 * rows * case["rank"] * (K + N)
    return {"bytes": nbytes, "flops": flops}


# -------------------------------------------------------------------- inputs

def _ints(values, dtype=torch.int32):
    return torch.tensor(list(values), dtype=dtype, device=DEVICE)


def _floats(values):
    return torch.tensor(list(values), dtype=torch.float32, device=DEVICE)


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    s = dict(case)
    if case["op"] == "sample":
        b, v = case["batch"], case["vocab"]
        # a trained model's logits: a broad middle, a few tokens above it, far or not, as sure as the model is
        z = torch.empty(b, v, device=DEVICE).normal_(0, 2.2, generator=g)
        top = torch.empty(b, v, device=DEVICE).exponential_(generator=g)
        z += 5.0 * torch.rand(b, 1, generator=g, device=DEVICE) * (top - 0.75 * math.log(v)).clamp(min=0)
        if case["masked"]:
            z.masked_fill_(torch.rand(b, v, generator=g, device=DEVICE) < case["masked"], -math.inf)
        s["z"] = z.to(torch.float16 if case["logits"] == "fp16" else torch.float32)
        t, k, p, m = zip(*_batch_settings(case))
        s["temperature"], s["top_k"], s["top_p"], s["min_p"] = _floats(t), _ints(k), _floats(p), _floats(m)
        s["noise"] = None
        if case["draw"]:
            s["noise"] = torch.empty(b, v, device=DEVICE).exponential_(generator=g).clamp_(min=1e-20)
        return s
    if case["op"] == "plan":
        got, free = _requests(case)
        n, new, held = zip(*got)
        page = case["page"]
        most = max(max(held), max(-(-(a + c) // page) for a, c in zip(n, new))) + 1
        pages = sum(held) + free
        order = torch.randperm(pages, generator=g, device=DEVICE).to(torch.int32)
        first = _ints([0] + list(held)).cumsum(0)[:-1]
        at = torch.arange(most, device=DEVICE)
        inside = at[None] < _ints(held)[:, None]
        s["table"] = torch.where(inside, order[(first[:, None] + at[None]).clamp(max=pages - 1)], -1).contiguous()
        s["lens"], s["new"], s["held"] = _ints(n), _ints(new), _ints(held)
        s["free_pages"] = torch.full((pages,), -1, dtype=torch.int32, device=DEVICE)
        s["free_pages"][:free] = order[sum(held):]
        s["free_count"] = _ints([free])
        s["rows"] = sum(new) + 3                        # a few rows of padding
        return s
    lens, which, rank = _rows_of(case), _adapters_of(case), case["rank"]
    s["cu"] = _ints([0] + lens).cumsum(0).to(torch.int32)
    s["adapter"] = _ints(which)
    s["scale"] = _floats(0.5 + 1.5 * random.Random(seed).random() for _ in range(case["adapters"]))
    s["x"], s["y"], s["A"], s["B"] = [], [], [], []
    for K, N in _shapes(case):
        x = torch.empty(case["rows"], K, dtype=torch.float16, device=DEVICE).normal_(generator=g)
        loud = torch.rand(K, generator=g, device=DEVICE) > 0.99     # channels that are large in every token
        s["x"].append(x * (1 + 9 * loud).half())
        s["y"].append(torch.empty(case["rows"], N, dtype=torch.float16, device=DEVICE).normal_(generator=g))
        s["A"].append(torch.empty(case["adapters"], rank, K, dtype=torch.float16, device=DEVICE)
                      .normal_(0, K ** -0.5, generator=g))
        s["B"].append(torch.empty(case["adapters"], N, rank, dtype=torch.float16, device=DEVICE)
                      .normal_(0, 0.3 * rank ** -0.5, generator=g))
    return s


# ----------------------------------------------------------------------- run

def run(s):
    if s["op"] == "sample":
        return _own_sample(s) if own else _plain_sample(s)
    if s["op"] == "plan":
        return _own_plan(s) if own else _plain_plan(s)
    return _own_adapters(s) if own else _plain_adapters(s)


def _own_sample(s):
    import w4_gemm_gated_amd as sp
    tokens, probs = sp.spear_sample(s["z"], s["noise"], temperature=s["temperature"], top_k=s["top_k"],
                                    top_p=s["top_p"], min_p=s["min_p"], probs=s["probs"])
    return {n: x for n, x in (("tokens", tokens), ("probs", probs)) if x is not None}


def _own_plan(s):
    import w4_gemm_gated_amd as sp
    cu, kv_lens, slots, positions, sequence, held, count = sp.spear_kv_plan(
        s["lens"], s["new"], s["held"], s["table"], s["free_pages"], s["free_count"], s["rows"], page_size=s["page"])
    return {"cu": cu, "kv_lens": kv_lens, "slots": slots, "positions": positions, "sequence": sequence, "held": held,
            "count": count, "table": s["table"], "free_pages": s["free_pages"]}


def _own_adapters(s):
    import w4_gemm_gated_amd as sp
    plan = sp.spear_adapter_plan(s["cu"], s["adapter"], s["adapters"], s["rows"])
    return [sp.spear_adapter_add(y, x, A, B, plan, scale=s["scale"])
            for y, x, A, B in zip(s["y"], s["x"], s["A"], s["B"])]


def _plain_sample(s):
    """Weights exp((z - max z) / T) and their sums in 64 bits, where a sum decides which
    token is the last that may be drawn.  Tokens in falling order of z, the lower index
    first: top-k keeps the first k, top-p the shortest run that holds p of what
    top-k left, min-p those of at least m times the largest weight."""
    z, v = s["z"], s["vocab"]
    order = torch.sort(z.float(), dim=-1, descending=True, stable=True)
    greedy = s["temperature"] <= 0
    t = torch.where(greedy, 1.0, s["temperature"]).double()[:, None]
    w = torch.exp((order.values - order.values[:, :1]).double() / t)      # the largest first: 1
    w = torch.where(w >= 2.0 ** -126, w, 0.0)
    place = torch.arange(v, device=z.device)[None]
    k = torch.where((s["top_k"] > 0) & ~greedy, s["top_k"], v)[:, None]
    k = torch.where(greedy[:, None], 1, k)
    left = torch.where(place < k, w, 0.0)
    before = left.cumsum(-1) - left
    p = s["top_p"].double()[:, None]
    kept = (left >= s["min_p"].double()[:, None]) & (left > 0)
    kept &= (before < p * left.sum(-1, keepdim=True)) | (p >= 1) | (place == 0)
    w = torch.where(kept, w, 0.0)
    got = {}
    if s["draw"]:
        noise = s["noise"].gather(-1, order.indices)
        score = torch.where(kept, w.float() / noise, -1.0)
        top = score.amax(-1, keepdim=True)
        got["tokens"] = torch.where(score == top, order.indices, v).amin(-1).to(torch.int32)
    if s["probs"]:
        w = (w / w.sum(-1, keepdim=True)).float()
        got["probs"] = torch.empty_like(w).scatter_(-1, order.indices, w)
    return got


def _plain_plan(s):
    page, rows = s["page"], s["rows"]
    lens, new, held = s["lens"].long(), s["new"].long(), s["held"].long()
    last = s["free_count"].long()                                       # pages on the stack
    most = s["table"].shape[1]
    want = (lens + new + page - 1) // page
    fits = (want <= most) & (held * page >= lens)
    freed = torch.where(fits, (held - want).clamp(min=0), 0)
    need = torch.where(fits, (want - held).clamp(min=0), 0)
    ask = torch.where(fits, new, 0)
    given = fits & (need.cumsum(0) <= last + freed.sum()) & (ask.cumsum(0) <= rows)
    n, take = torch.where(given, new, 0), torch.where(given, need, 0)
    cu = torch.cat([torch.zeros_like(last), n.cumsum(0)])
    kv_lens, now = lens + n, held - freed + take
    # the stack: what is let go is laid on it in order, what is taken comes from its top
    at = torch.arange(most, device=lens.device)[None]
    old, b_freed = s["table"], (at >= (held - freed)[:, None]) & (at < held[:, None])
    stack = torch.cat([s["free_pages"].long(), torch.zeros(rows, dtype=torch.long, device=lens.device)])
    first_freed = freed.cumsum(0) - freed + last
    place = torch.where(b_freed, first_freed[:, None] + at - (held - freed)[:, None], stack.numel() - 1)
    full = stack.scatter(0, place.flatten(), torch.where(b_freed, old, 0).long().flatten())
    first = take.cumsum(0) - take
    taken = (at >= held[:, None]) & (at < (held + take)[:, None])
    top = (last + freed.sum() - 1 - first[:, None] - (at - held[:, None])).clamp(min=0, max=stack.numel() - 1)
    table = torch.where(taken, full[top], old.long())
    s["table"].copy_(table)
    count = last + freed.sum() - take.sum()
    at = torch.arange(s["free_pages"].numel(), device=lens.device)
    s["free_pages"].copy_(torch.where((at >= last) & (at < count), full[:at.numel()], s["free_pages"].long()))
    row = torch.arange(rows, device=lens.device)
    b = torch.bucketize(row, cu[1:].contiguous(), right=True).clamp(max=lens.numel() - 1)
    used = row < cu[-1]
    pos = lens[b] + row - cu[b]
    slot = table[b, (pos // page).clamp(max=most - 1)] * page + pos % page
    i32 = lambda x: x.to(torch.int32)  # noqa: E731
    return {"cu": i32(cu), "kv_lens": i32(kv_lens), "slots": torch.where(used, slot, -1),
            "positions": i32(torch.where(used, pos, -1)), "sequence": i32(torch.where(used, b, -1)), "held": i32(now),
            "count": i32(count), "table": s["table"], "free_pages": s["free_pages"]}


def _plain_add(y, x, A, B, of, scale):
    """y + scale[a] (x A[a]') B[a]' with a = of[row]: all adapters' products, the row's own kept."""
    n, rank, K = A.shape
    h = torch.matmul(x.float(), A.float().view(n * rank, K).t()).view(-1, n, rank)
    mine = of[:, None] == torch.arange(n, device=of.device)[None]
    h = torch.where(mine[..., None], h * scale[None, :, None], 0.0)
    d = torch.matmul(h.view(-1, n * rank), B.float().transpose(1, 2).reshape(n * rank, -1))
    y.copy_(torch.where((of >= 0)[:, None], (y.float() + d).half(), y))
    return y


def _plain_adapters(s):
    row = torch.arange(s["rows"], device=s["cu"].device)
    of = s["adapter"].long()[torch.bucketize(row, s["cu"][1:].long(), right=True)]
    return [_plain_add(y, x, A, B, of, s["scale"]) for y, x, A, B in zip(s["y"], s["x"], s["A"], s["B"])]


# --------------------------------------------------------------------- exact

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "plan":
        return None                                     # whole numbers only
    if case["op"] == "sample":
        if not case["probs"]:
            return None
        got = {"tokens": None} if case["draw"] else {}
        probs = torch.zeros(case["batch"], case["vocab"], dtype=torch.float64, device=DEVICE)
        for b, (t, k, p, m) in enumerate(zip(*(s[n].tolist() for n in ("temperature", "top_k", "top_p", "min_p")))):
            z = s["z"][b].double()
            by = torch.argsort(-z, stable=True)[:int((z > -math.inf).sum())]
            if t <= 0:
                probs[b, by[0]] = 1.0
                continue
            by = by[:int(k)] if k > 0 else by
            share = torch.softmax(z[by] / t, -1)
            run_to = share.cumsum(-1) - share
            last = max(1, int((run_to < p).sum())) if p < 1 else by.numel()
            last = min(last, int((share >= m * share[0]).sum()))
            probs[b, by[:last]] = share[:last] / share[:last].sum()
        got["probs"] = probs
        return got
    got, cu = [], s["cu"].tolist()
    for y, x, A, B in zip(s["y"], s["x"], s["A"], s["B"]):
        y = y.double()
        for b, a in enumerate(s["adapter"].tolist()):
            if a >= 0:
                at = slice(cu[b], cu[b + 1])
                y[at] += float(s["scale"][a]) * (x[at].double() @ A[a].double().T @ B[a].double().T)
        got.append(y)
    return got

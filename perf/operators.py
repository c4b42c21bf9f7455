"""Workloads of the serving operators beside the W4 linear layer: the paged
key/value cache (written in fp16 or quantised to 8 bits, and read back),
attention of new tokens over that cache, and the verification of drafted
tokens.

Each case is run either in its plain form (elementary torch operations in 32
bits) or, with `own` set, by the calls a user makes of the framework.

The cache: pages [num_pages, kv_heads, page_size, head_dim]; token i of a
sequence lies in page block_table[b, i // page_size], place i % page_size.  The
8-bit form keeps one fp32 scale per token and head, s = max|x| / 127, and
codes rint(x / s).
"""
import math
import random

import torch

own = False

DEVICE = "cuda"


# --------------------------------------------------------------------- cases

def listed():
    return [
        # One new token for each of a few short sequences, 16 heads of 128
        # over a hidden width of 2048: a lightly loaded server, latency counts.
        dict(name="decode_small", op="attention", cache="fp16", batch=4, kv_min=90, kv_max=700, q_min=1, q_max=1,
             chunks=0, chunk=0, q_heads=16, kv_heads=16, head_dim=128, page=16, lens=1),
        # Decode of a full batch with very different lengths (width 4096, keys
        # and values 1024 wide), 8-bit cache: the ordinary serving step.
        dict(name="decode_batch_int8", op="attention", cache="int8", batch=96, kv_min=64, kv_max=8192, q_min=1,
             q_max=1, chunks=0, chunk=0, q_heads=32, kv_heads=8, head_dim=128, page=32, lens=2),
        # Two long contexts and nothing else to fill the GPU with.
        dict(name="decode_long", op="attention", cache="fp16", batch=2, kv_min=50001, kv_max=70001, q_min=1,
             q_max=1, chunks=0, chunk=0, q_heads=32, kv_heads=8, head_dim=128, page=64, lens=3),
        # Each sequence's last token and up to five drafted ones.
        dict(name="draft_int8", op="attention", cache="int8", batch=24, kv_min=500, kv_max=6000, q_min=1, q_max=6,
             chunks=0, chunk=0, q_heads=32, kv_heads=8, head_dim=128, page=16, lens=4),
        # A 2048-token chunk of a long prompt, the rest already cached.
        dict(name="chunk", op="attention", cache="fp16", batch=1, kv_min=8192, kv_max=8192, q_min=2048, q_max=2048,
             chunks=0, chunk=0, q_heads=32, kv_heads=8, head_dim=128, page=64, lens=5),
        # A prompt's chunk in one batch with the decode steps of 40 others.
        dict(name="mixed_int8_d64", op="attention", cache="int8", batch=41, kv_min=200, kv_max=5000, q_min=1,
             q_max=1, chunks=1, chunk=700, q_heads=32, kv_heads=8, head_dim=64, page=16, lens=6),
        # A decode step's new keys and values, some rows padding (slot -1).
        dict(name="write_step", op="cache", cache="fp16", what="write", batch=48, kv_min=1, kv_max=512, kv_heads=8,
             head_dim=128, page=16, lens=7),
        # Prompts written to the 8-bit cache and read back for a consumer
        # that wants them whole.
        dict(name="write_read_int8", op="cache", cache="int8", what="write_read", batch=5, kv_min=300, kv_max=4001,
             kv_heads=8, head_dim=128, page=32, lens=8),
        # Reading long 8-bit sequences back.
        dict(name="read_int8", op="cache", cache="int8", what="read", batch=24, kv_min=1000, kv_max=9000, kv_heads=8,
             head_dim=128, page=64, lens=9),
        # One or two users, few drafts: latency.
        dict(name="verify_small", op="verify", batch=2, drafts=3, vocab=32000, given=True, lens=10),
        # A full batch over a large vocabulary.
        dict(name="verify_batch", op="verify", batch=64, drafts=5, vocab=128001, given=True, lens=11),
        # Drafts copied from the prompt: no draft probabilities.
        dict(name="verify_copied", op="verify", batch=24, drafts=8, vocab=50257, given=False, lens=12),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def _draw_any(rng):
    op = rng.choice(["attention", "attention", "cache", "verify"])
    lens = rng.randrange(1, 1 << 30)
    if op == "verify":
        return dict(op=op, batch=_log_int(rng, 1, 64), drafts=rng.randint(1, 8), vocab=_log_int(rng, 30000, 130000),
                    given=rng.random() < 0.7, lens=lens)
    heads = dict(kv_heads=rng.choice([2, 4, 8, 16]), head_dim=rng.choice([64, 128]), page=rng.choice([16, 32, 64]),
                 cache=rng.choice(["fp16", "int8"]), lens=lens)
    if op == "cache":
        lo = _log_int(rng, 1, 2000)
        return dict(op=op, what=rng.choice(["write", "write_read", "read"]) if heads["cache"] == "int8" else "write",
                    batch=_log_int(rng, 1, 64), kv_min=lo, kv_max=_log_int(rng, lo, 9000), **heads)
    heads["q_heads"] = heads["kv_heads"] * rng.choice([1, 2, 4, 8])
    kind = rng.choice(["decode", "draft", "chunk", "mixed"])
    lo = _log_int(rng, 60, 50000)
    c = dict(op=op, batch=_log_int(rng, 1, 96), kv_min=lo, kv_max=_log_int(rng, lo, 70000), q_min=1, q_max=1,
             chunks=0, chunk=0, **heads)
    if kind == "draft":
        c["q_max"] = rng.randint(2, 9)
    if kind == "chunk":
        c["batch"] = rng.randint(1, 4)
        c["q_max"] = _log_int(rng, 33, 2048)
        c["q_min"] = _log_int(rng, 17, c["q_max"])
    if kind == "mixed":
        c["chunks"] = rng.randint(1, 2)
        c["batch"] += c["chunks"]
        c["chunk"] = _log_int(rng, 65, 1024)
    return c


def draw(rng):
    most = max(_cost(c) for c in listed())
    least = min(_cost(c) for c in listed())
    while True:
        c = _draw_any(rng)
        if least <= _cost(c) <= most and _plain_bytes(c) <= 24e9:
            return c


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def _lengths(case):
    """(new tokens, cached tokens with them) of each sequence, by the case."""
    r = random.Random(case["lens"])
    kv = [_log_int(r, case["kv_min"], case["kv_max"]) for _ in range(case["batch"])]
    if case["op"] == "cache":
        return kv, kv
    q = [r.randint(case["q_min"], case["q_max"]) for _ in range(case["batch"])]
    for b in range(case["chunks"]):
        q[b] = case["chunk"]
    return q, [max(a, b) for a, b in zip(q, kv)]


def _plain_bytes(case):
    """Memory of the plain attention's padded tensors."""
    if case["op"] != "attention":
        return 0
    q, kv = _lengths(case)
    pairs = case["batch"] * max(kv)
    return pairs * (4.0 * case["q_heads"] * max(q) * 2 + 4.0 * case["kv_heads"] * case["head_dim"] * 4)


def work(case):
    if case["op"] == "verify":
        b, k, v = case["batch"], case["drafts"], case["vocab"]
        # per sequence: the drafted entries, then one row each of target
        # probabilities, noise and (if given) draft probabilities
        rows = 3 if case["given"] else 2
        return {"bytes": 4.0 * (b * rows * v + b * k * 4 + b * (k + 2)), "flops": 3.0 * b * v}
    h, d = case["kv_heads"], case["head_dim"]
    q, kv = _lengths(case)
    held = 2 * h * (d * 2 if case["cache"] == "fp16" else d + 4)    # one cached token, keys and values
    given = 2 * h * d * 2                                           # the same token in fp16
    if case["op"] == "cache":
        written = {"write": case["batch"], "write_read": sum(kv), "read": 0}[case["what"]]
        read = 0 if case["what"] == "write" and case["cache"] == "fp16" else sum(kv)
        return {"bytes": float(written * (given + held + 8) + read * (held + given)),
                "flops": float(2 * h * d * (2 * written + read))}
    pairs = sum(a * b - a * (a - 1) // 2 for a, b in zip(q, kv))
    rows = sum(q) * case["q_heads"] * d * 2
    return {"bytes": float(sum(kv) * held + 2 * rows + 4 * sum(-(-n // case["page"]) for n in kv)),
            "flops": 4.0 * d * case["q_heads"] * pairs}


# -------------------------------------------------------------------- inputs

def _table(case, kv, g):
    """Pages of every sequence in random places: (block_table, pages in all)."""
    page = case["page"]
    n = [-(-x // page) for x in kv]
    total = sum(n) + 3
    order = torch.randperm(total, generator=g, device=DEVICE, dtype=torch.int64).to(torch.int32)
    first = torch.tensor([0] + n, device=DEVICE).cumsum(0)[:-1]
    at = torch.arange(max(n), device=DEVICE)
    held = torch.tensor(n, device=DEVICE)
    table = torch.where(at[None] < held[:, None], order[(first[:, None] + at[None]).clamp(max=total - 1)], -1)
    return table.to(torch.int32).contiguous(), total


def _cu(lens):
    return torch.tensor([0] + list(lens), device=DEVICE).cumsum(0).to(torch.int32)


def _cache(case, pages, g):
    shape = (pages, case["kv_heads"], case["page"], case["head_dim"])
    got = {}
    # keys have a few channels that are large in every token, as trained ones do
    loud = 1 + 4 * (torch.rand(case["kv_heads"], 1, case["head_dim"], generator=g, device=DEVICE) > 0.97).half()
    for n in ("k", "v"):
        if case["cache"] == "fp16":
            x = torch.empty(shape, dtype=torch.float16, device=DEVICE).normal_(generator=g)
            got[n + "_cache"] = x.mul_(loud) if n == "k" else x
            got[n + "_scale"] = None
        else:
            x = torch.empty(shape, dtype=torch.float16, device=DEVICE).normal_(0, 40, generator=g)
            got[n + "_cache"] = x.round_().clamp_(-127, 127).to(torch.int8)
            s = torch.empty(shape[:3], dtype=torch.float32, device=DEVICE).normal_(generator=g)
            got[n + "_scale"] = s.mul_(0.25).exp_().mul_(0.025)
    return got


def prepare(case, seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)
    s = dict(case)
    if case["op"] == "verify":
        b, k, v = case["batch"], case["drafts"], case["vocab"]
        logits = torch.empty(b, k + 1, v, device=DEVICE).normal_(0, 2.5, generator=g)
        s["target"] = torch.softmax(logits, -1)
        near = logits[:, :k] + torch.empty(b, k, v, device=DEVICE).normal_(0, 0.7, generator=g)
        near = torch.softmax(near, -1)
        race = torch.empty(b, k, v, device=DEVICE).exponential_(generator=g)
        s["drafted"] = (near / race).argmax(-1).to(torch.int32)
        if not case["given"]:   # a copied token is often the target's best
            best = logits[:, :k].argmax(-1).to(torch.int32)
            s["drafted"] = torch.where(torch.rand(b, k, generator=g, device=DEVICE) < 0.7, best, s["drafted"])
        s["draft"] = near if case["given"] else None
        s["u"] = torch.rand(b, k, generator=g, device=DEVICE)
        s["noise"] = torch.empty(b, v, device=DEVICE).exponential_(generator=g).clamp_(min=1e-20)
        r = random.Random(case["lens"])
        n = [k] + [r.randint(0, k) if r.random() < 0.3 else k for _ in range(b - 1)]
        s["drafts_of"] = torch.tensor(n, dtype=torch.int32, device=DEVICE)
        return s
    q, kv = _lengths(case)
    s["max_q"], s["max_kv"], s["total"] = max(q), max(kv), sum(q)
    s["table"], pages = _table(case, kv, g)
    s.update(_cache(case, pages, g))
    h, d = case["kv_heads"], case["head_dim"]
    s["kv_lens"] = torch.tensor(kv, dtype=torch.int32, device=DEVICE)
    if case["op"] == "attention":
        s["cu_q"] = _cu(q)
        # the queries as they lie in a joint projection's output
        joint = torch.empty(sum(q), (case["q_heads"] + 2 * h) * d, dtype=torch.float16, device=DEVICE)
        joint.normal_(0, 1.3, generator=g)
        s["q"] = joint[:, :case["q_heads"] * d].view(sum(q), case["q_heads"], d)
        return s
    s["cu_kv"] = _cu(kv)
    rows = case["batch"] if case["what"] == "write" else sum(kv)
    joint = torch.empty(rows, 4 * h * d, dtype=torch.float16, device=DEVICE).normal_(generator=g)
    s["k"] = joint[:, 2 * h * d:3 * h * d].view(rows, h, d)
    s["v"] = joint[:, 3 * h * d:].view(rows, h, d)
    if case["what"] == "write":     # the last token of every sequence; every fifth row is padding
        b = torch.arange(rows, device=DEVICE)
        at = s["kv_lens"].long() - 1
        place = s["table"][b, at // case["page"]].long() * case["page"] + at % case["page"]
        s["slots"] = torch.where(b % 5 == 4, -1, place)
    else:
        b, at = _rows_of(s["cu_kv"], rows)
        s["slots"] = s["table"][b, at // case["page"]].long() * case["page"] + at % case["page"]
    return s


def _rows_of(cu, total):
    """(sequence, place in it) of each of the `total` rows."""
    row = torch.arange(total, device=cu.device)
    b = torch.bucketize(row, cu[1:].long(), right=True)
    return b, row - cu[b].long()


# ----------------------------------------------------------------------- run

def run(s):
    if s["op"] == "attention":
        return _own_attention(s) if own else _plain_attention(s)
    if s["op"] == "cache":
        return _own_cache(s) if own else _plain_cache(s)
    return _own_verify(s) if own else _plain_verify(s)


def _own_attention(s):
    import w4_gemm_gated_amd as sp
    return sp.spear_paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"], s["cu_q"], s["kv_lens"],
                                    s["max_q"], k_scale=s["k_scale"], v_scale=s["v_scale"])


def _own_cache(s):
    import w4_gemm_gated_amd as sp
    if s["what"] != "read":
        sp.spear_kv_append(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"], k_scale=s["k_scale"],
                           v_scale=s["v_scale"])
    if s["what"] == "write" and s["cache"] == "fp16":
        return {"k": s["k_cache"], "v": s["v_cache"]}
    k, v = sp.spear_kv_gather(s["k_cache"], s["v_cache"], s["table"], s["cu_kv"], s["total"], k_scale=s["k_scale"],
                              v_scale=s["v_scale"])
    return {"k": k, "v": v, "k_scale": s["k_scale"], "v_scale": s["v_scale"]}


def _own_verify(s):
    import w4_gemm_gated_amd as sp
    return sp.spear_verify_draft(s["target"], s["draft"], s["drafted"], s["u"], s["noise"], num_drafts=s["drafts_of"])


def _pages(cache, scale, table):
    """The cached tokens of every sequence in 32 bits: [B, heads, tokens, head_dim]."""
    t = table.clamp(min=0).long()
    x = cache[t].float()
    if scale is not None:
        x = x * scale[t][..., None]
    b, p, h, n, d = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(b, h, p * n, d)


def _plain_attention(s):
    h, d, most = s["kv_heads"], s["head_dim"], s["max_q"]
    group = s["q_heads"] // h
    k, v = (_pages(s[n + "_cache"], s[n + "_scale"], s["table"]) for n in ("k", "v"))
    cu, kv = s["cu_q"].long(), s["kv_lens"].long()
    new = cu[1:] - cu[:-1]
    at = torch.arange(most, device=cu.device)
    rows = (cu[:-1, None] + at[None]).clamp(max=s["total"] - 1)                             # [B, most]
    q = s["q"][rows].float().view(-1, most, h, group, d).permute(0, 2, 1, 3, 4).reshape(-1, h, most * group, d)
    score = torch.matmul(q, k.transpose(-1, -2).contiguous()) * (1.0 / math.sqrt(d))
    last = kv[:, None] - new[:, None] + at[None]                                            # last visible key
    key = torch.arange(k.shape[2], device=cu.device)
    seen = (key[None, None] <= last[..., None]) & (key[None, None] < kv[:, None, None])     # [B, most, keys]
    seen = seen.repeat_interleave(group, 1)[:, None]
    score = torch.where(seen, score, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(torch.isinf(top), 0.0, top))
    out = torch.matmul(p, v)
    total = p.sum(-1, keepdim=True)
    out = torch.where(total > 0, out / total, 0.0)
    out = out.view(-1, h, most, group, d).permute(0, 2, 1, 3, 4).reshape(-1, most, s["q_heads"], d)
    b, i = _rows_of(s["cu_q"], s["total"])
    return out[b, i].to(torch.float16)


def _plain_write(s, n):
    x, page = s[n], s["page"]
    row = (s["slots"] >= 0).nonzero()[:, 0]
    x, slot = x[row].float(), s["slots"][row]
    if s["cache"] == "int8":
        most = x.abs().amax(-1)
        scale = most / torch.full_like(most, 127.0)
        x = torch.where(scale[..., None] > 0, torch.round(x / scale[..., None]), 0.0).clamp(-127, 127)
        s[n + "_scale"][slot // page, :, slot % page] = scale
    s[n + "_cache"][slot // page, :, slot % page] = x.to(s[n + "_cache"].dtype)


def _plain_cache(s):
    if s["what"] != "read":
        _plain_write(s, "k")
        _plain_write(s, "v")
    if s["what"] == "write" and s["cache"] == "fp16":
        return {"k": s["k_cache"], "v": s["v_cache"]}
    b, at = _rows_of(s["cu_kv"], s["total"])
    page, place = s["table"][b, at // s["page"]].long(), at % s["page"]
    got = {"k_scale": s["k_scale"], "v_scale": s["v_scale"]}
    got |= {n: (s[n + "_cache"][page, :, place].float() * s[n + "_scale"][page, :, place][..., None]).half()
            for n in ("k", "v")}
    return got


def _plain_verify(s):
    k, v = s["drafts"], s["vocab"]
    n = s["drafts_of"].long()
    at = torch.arange(k, device=n.device)
    x = s["drafted"].long()
    p = s["target"][:, :k].gather(-1, x[..., None])[..., 0]
    q = s["draft"].gather(-1, x[..., None])[..., 0] if s["draft"] is not None else torch.ones_like(p)
    ok = (s["u"] * q < p) & (at[None] < n[:, None])
    kept = ok.long().cumprod(1).sum(1)                                   # accepted drafts
    b = torch.arange(n.numel(), device=n.device)
    target = s["target"][b, kept]
    stop = kept.clamp(max=k - 1)
    if s["draft"] is not None:
        other = s["draft"][b, stop]
    else:
        other = (torch.arange(v, device=n.device)[None] == x[b, stop][:, None]).float()
    rest = (target - other).clamp(min=0)
    use = (kept < n) & (rest > 0).any(-1)
    weight = torch.where(use[:, None], rest, target)
    score = torch.where(weight > 0, weight / s["noise"], -1.0)
    top = score.amax(-1, keepdim=True)
    token = torch.where(score == top, torch.arange(v, device=n.device)[None], v).amin(-1)
    at = torch.arange(k + 1, device=n.device)[None]
    drafted = torch.cat([x, x[:, :1]], 1)
    tokens = torch.where(at < kept[:, None], drafted, torch.where(at == kept[:, None], token[:, None], -1))
    return kept.to(torch.int32), tokens.to(torch.int32)


# --------------------------------------------------------------------- exact

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attention":
        return _exact_attention(s)
    if case["op"] == "cache":
        return _exact_cache(s)
    return None     # whole numbers only


def _exact_tokens(s, n, b, length):
    """Keys or values of one sequence in 64 bits: [heads, length, head_dim]."""
    page = s["page"]
    ids = s["table"][b, :-(-length // page)].long()
    x = s[n + "_cache"].index_select(0, ids).double()
    if s[n + "_scale"] is not None:
        x *= s[n + "_scale"].index_select(0, ids).double().unsqueeze(-1)
    return x.transpose(0, 1).flatten(1, 2)[:, :length]


def _exact_attention(s):
    out = torch.zeros(s["total"], s["q_heads"], s["head_dim"], dtype=torch.float64, device=DEVICE)
    cu, lens = s["cu_q"].tolist(), s["kv_lens"].tolist()
    group = s["q_heads"] // s["kv_heads"]
    for b, length in enumerate(lens):
        k, v = _exact_tokens(s, "k", b, length), _exact_tokens(s, "v", b, length)
        for at in range(cu[b], cu[b + 1], 512):
            end = min(cu[b + 1], at + 512)
            place = length - (cu[b + 1] - torch.arange(at, end, device=DEVICE))     # position of each row
            hidden = torch.arange(length, device=DEVICE)[None] > place[:, None]
            for head in range(s["q_heads"]):
                z = s["q"][at:end, head].double() @ k[head // group].T / math.sqrt(s["head_dim"])
                z.masked_fill_(hidden, -math.inf)
                out[at:end, head] = torch.softmax(z, -1) @ v[head // group]
    return out


def _exact_cache(s):
    page = s["page"]
    if s["what"] == "write" and s["cache"] == "fp16":
        got = {}
        for n in ("k", "v"):
            whole = s[n + "_cache"].double()
            for row, slot in enumerate(s["slots"].tolist()):
                if slot >= 0:
                    whole[slot // page, :, slot % page] = s[n][row].double()
            got[n] = whole
        return got
    got = {}
    if s["what"] == "read":
        for n in ("k", "v"):
            got[n] = torch.cat([_exact_tokens(s, n, b, m).transpose(0, 1) for b, m in enumerate(s["kv_lens"].tolist())])
            got[n + "_scale"] = s[n + "_scale"].double()
        return got
    for n in ("k", "v"):
        # what the codes stand for is compared with no tie broken another way
        row = (s["slots"] >= 0).nonzero()[:, 0]
        x = s[n].double()
        scale = s[n + "_scale"].double()
        slot = s["slots"][row]
        scale[slot // page, :, slot % page] = x[row].abs().amax(-1) / 127
        got[n + "_scale"], got[n] = scale, None
    return got

"""Speculative decoding with W4 layers and a paged 8-bit cache, on one GPU.

A one-layer causal language model (random weights): embedding, W4 + EC joint
projection to queries, keys and values, attention over the paged cache, W4 + EC
output projection, W4 head.  The target runs it with the error compensators on;
the drafter is the same model with them switched off, which costs less a call and
mostly agrees.  Each round the drafter proposes `drafts` tokens one at a time, the
target scores all of them in one call (a chunk of new tokens over its cache),
and the verification keeps those that leave the output distributed as the
target's.  Both draw from the same rules (temperature, top-p).  Rejected tokens stay
in the cache's memory and are written over; pages that no sequence needs any more go
back to the free ones with the next step's plan.

    python examples/speculative_decoding.py --rounds 8
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import w4_gemm_gated_amd as sp  # noqa: E402

PAGE = 16


class Linear:
    """A W4 linear with an error compensator initialised from its residual."""

    def __init__(self, K, N, rank, g):
        W = torch.empty(K, N, dtype=torch.float16, device="cuda").normal_(0, K ** -0.5, generator=g)
        self.Wq, self.s = sp.spear_pack_w4(W)
        self.A, self.B = sp.spear_ec_init(W, self.Wq, self.s, rank)
        self.w_g = torch.zeros(K, dtype=torch.float16, device="cuda")

    def __call__(self, x, ec):
        # a gate bias of 4 keeps the compensator almost fully on
        return sp.spear_w4ec_linear(x.contiguous(), self.Wq, self.s, self.A, self.B, self.w_g, 4.0,
                                    variant="auto" if ec else "no_ec")


def norm(x):
    return (x.float() * torch.rsqrt(x.float().pow(2).mean(-1, keepdim=True) + 1e-6)).half()


class Model:
    def __init__(self, vocab, hidden, q_heads, kv_heads, dim, g):
        self.vocab, self.q_heads, self.kv_heads, self.dim = vocab, q_heads, kv_heads, dim
        self.embed = torch.empty(vocab, hidden, dtype=torch.float16, device="cuda").normal_(generator=g)
        self.qkv = Linear(hidden, (q_heads + 2 * kv_heads) * dim, 16, g)
        self.out = Linear(q_heads * dim, hidden, 16, g)
        self.head = Linear(hidden, vocab, 16, g)

    def __call__(self, tokens, seqs, cu, max_new, ec):
        """Logits of every new token; their keys and values enter the cache first.
        tokens: the batch's new tokens one sequence after the other, cu[b] ..
        cu[b + 1] - 1 those of sequence b, already counted in seqs.lens."""
        h, kv, d = self.q_heads, self.kv_heads, self.dim
        x = self.embed[tokens]
        y = self.qkv(norm(x), ec)
        q = y[:, :h * d].view(-1, h, d)
        k = y[:, h * d:(h + kv) * d].view(-1, kv, d)
        v = y[:, (h + kv) * d:].view(-1, kv, d)
        sp.spear_kv_append(k, v, seqs.slots(cu, tokens.numel()), *seqs.cache)
        o = sp.spear_paged_attention(q, seqs.cache[0], seqs.cache[1], seqs.table, cu, seqs.lens, max_new,
                                     k_scale=seqs.cache[2], v_scale=seqs.cache[3])
        x = x + self.out(o.view(-1, h * d), ec)
        return self.head(norm(x), ec)


class Sequences:
    """A batch's paged cache: pages are taken from a stack of free ones in random order."""

    def __init__(self, batch, room, model, g, dtype=torch.int8):
        most = -(-room // PAGE)
        self.cache = sp.spear_kv_cache(batch * most, model.kv_heads, model.dim, PAGE, dtype)
        self.free_pages = torch.randperm(batch * most, generator=g, device="cuda").to(torch.int32)
        self.free_count = torch.full((1,), batch * most, dtype=torch.int32, device="cuda")
        self.table = torch.zeros(batch, most, dtype=torch.int32, device="cuda")
        self.held = torch.zeros(batch, dtype=torch.int32, device="cuda")
        self.lens = torch.zeros(batch, dtype=torch.int32, device="cuda")

    def slots(self, cu, rows):
        """Where the last cu[b + 1] - cu[b] tokens of each sequence lie, on new pages as
        far as it has none for them."""
        new = cu[1:] - cu[:-1]
        return sp.spear_kv_plan(self.lens - new, new, self.held, self.table, self.free_pages, self.free_count, rows,
                                page_size=PAGE, held_out=self.held, free_out=self.free_count)[2]


def offsets(n, batch):
    return torch.arange(batch + 1, dtype=torch.int32, device="cuda") * n


def generate(batch=4, prompt=50, rounds=8, drafts=4, temperature=0.3, vocab=1000, hidden=512, q_heads=8, kv_heads=2,
             dim=64, seed=0, dtype=torch.int8, top_p=0.95):
    """Runs `rounds` rounds; returns the model, the target's sequences, each
    sequence's tokens (lists, the prompt first) and the kept drafts per round."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    model = Model(vocab, hidden, q_heads, kv_heads, dim, g)
    room = prompt + (rounds + 1) * (drafts + 1)
    target, draft = (Sequences(batch, room, model, g, dtype) for _ in range(2))
    text = torch.randint(vocab, (batch, prompt), generator=g, device="cuda")
    tokens = [row.tolist() for row in text]

    def noise():
        return torch.empty(batch, vocab, device="cuda").exponential_(generator=g)

    rules = dict(temperature=temperature, top_p=top_p, probs=True)

    # The prompt, all but its last token, into both caches as one chunk.
    for seqs, ec in ((target, True), (draft, False)):
        seqs.lens += prompt - 1
        model(text[:, :-1].reshape(-1), seqs, offsets(prompt - 1, batch), prompt - 1, ec)
    last = text[:, -1].to(torch.int32)
    one, chunk = offsets(1, batch), offsets(drafts + 1, batch)
    kept = []
    for _ in range(rounds):
        # The drafter, one token at a time.
        start = draft.lens.clone()
        new, p_draft = [last], []
        for _ in range(drafts):
            draft.lens += 1
            drawn, p = sp.spear_sample(model(new[-1].long(), draft, one, 1, False), noise(), **rules)
            p_draft.append(p)
            new.append(drawn)
        draft.lens += 1                         # the last drafted token's keys, should it be kept
        model(new[-1].long(), draft, one, 1, False)
        new = torch.stack(new, 1)               # [batch, 1 + drafts]
        # The target, all of them at once.
        target.lens += drafts + 1
        _, p_target = sp.spear_sample(model(new.reshape(-1).long(), target, chunk, drafts + 1, True), **rules)
        accepted, out = sp.spear_verify_draft(
            p_target.view(batch, drafts + 1, vocab), torch.stack(p_draft, 1), new[:, 1:].contiguous(),
            torch.rand(batch, drafts, generator=g, device="cuda"), noise())
        # What was refused leaves the caches: the lengths go back.
        target.lens -= drafts - accepted
        draft.lens.copy_(start + 1 + accepted)
        last = out.gather(1, accepted[:, None].long())[:, 0]
        for b, row in enumerate(out.tolist()):
            tokens[b] += [t for t in row if t >= 0]
        kept.append(accepted.tolist())
    return model, target, tokens, kept


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--rounds", type=int, default=8)
    ap.add_argument("--batch", type=int, default=4)
    ap.add_argument("--drafts", type=int, default=4)
    a = ap.parse_args()
    _, _, tokens, kept = generate(batch=a.batch, rounds=a.rounds, drafts=a.drafts)
    for b, row in enumerate(tokens):
        print(f"sequence {b}: {row[50:]}")
    mean = sum(map(sum, kept)) / (len(kept) * a.batch)
    print(f"kept {mean:.2f} of {a.drafts} drafted tokens per round: {1 + mean:.2f} tokens for each target call")

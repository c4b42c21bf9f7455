"""Block tables, adapters and sampling run together with the W4 layers, the paged cache,
attention and verification, as a serving step uses them; and their calls beside the
others': one workspace for all, captured without one, on another device."""
import numpy as np
import pytest
import torch

import workloads
from oracle import spear_step as ref
import w4_gemm_gated_amd as sp
import test_gpu_adapter as ad
import test_gpu_kv_plan as kp
import test_gpu_sample as sa
from test_gpu_shared_workspace import attention, layer, verification

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]
DEV = "cuda:0"
I32 = dict(dtype=torch.int32, device=DEV)


def note(msg):
    print(f"[gpu-step] {msg}", flush=True)


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


# ------------------------------------------------------------- the calls alone

def planned(B=600, rows=1500):
    rng = np.random.default_rng(B)
    s = kp.state(rng, B, 16, 60, 4)
    t = [dev(np.asarray(x, np.int32)) for x in (s[0], s[1], s[2], s[3], s[4], [s[5]])]

    def call(ws=None):
        table, stack = t[3].clone(), t[4].clone()
        out = sp.spear_kv_plan(*t[:3], table, stack, t[5], rows, workspace=ws)
        return torch.cat([x.flatten().long() for x in (*out, table, stack)])
    return call


def adapted(lens, K, N, rank):
    rng = np.random.default_rng(K + N)
    cu, of, rows = ad.batch(rng, lens, 3)
    X, A, B, Y = ad.tensors(rng, rows, K, N, rank, 3)
    t = [dev(X), dev(A), dev(B)]
    y = dev(Y)
    plan = sp.spear_adapter_plan(dev(cu), dev(of), 3, rows)
    return lambda ws=None: sp.spear_adapter_add(y.clone(), *t, plan, workspace=ws)


def sampled(B, V):
    rng = np.random.default_rng(V)
    z, noise = dev(sa.logits(rng, B, V)), dev(rng.exponential(size=(B, V)).astype(np.float32))
    s = sa.settings([sa.RULES[b % len(sa.RULES)] for b in range(B)])

    def call(ws=None):
        tokens, probs = sp.spear_sample(z, noise, probs=True, workspace=ws, **s)
        return torch.cat([tokens.float(), probs.flatten()])
    return call


CALLS = {"block tables": planned, "adapters of single tokens": lambda: adapted([1] * 40, 1024, 700, 16),
         "adapters of long rows": lambda: adapted([1, 1, 200, 40], 8192, 512, 32),
         "draws": lambda: sampled(9, 50257), "draws of short rows": lambda: sampled(30, 900)}


@pytest.mark.parametrize("given", [True, False])
def test_all_operators_share_a_workspace(given, monkeypatch):
    """Every call gives the bits that it gives on a workspace of its own, in any order
    and with no wait between them."""
    note("given" if given else "the stream's")
    calls = {n: make() for n, make in CALLS.items()}
    calls.update({"split decode": layer(16, 2048, 1024, 32, "split"), "fused tiles": layer(200, 1024, 2048, 32, "fused"),
                  "decode": attention([1, 1, 1], [4000, 40, 900], True),
                  "chunk and decode": attention([300, 1], [2500, 3000], False), "verification": verification(3, 2, 50000)})
    monkeypatch.setattr(sp, "_workspaces", {})
    own = {n: call(torch.zeros(256 << 20, dtype=torch.uint8, device=DEV)).clone() for n, call in calls.items()}
    torch.cuda.synchronize()
    ws = torch.zeros(256 << 20, dtype=torch.uint8, device=DEV) if given else None
    rng = np.random.default_rng(8)
    order = [n for _ in range(6) for n in rng.permutation(list(calls))]
    got = [(n, calls[n](ws)) for n in order]
    torch.cuda.synchronize()
    for n, x in got:
        assert torch.equal(x, own[n]), n
    assert sp.spear_take_error(ws) == 0


@pytest.mark.parametrize("kind", CALLS)
def test_capture_without_a_workspace_is_refused(monkeypatch, kind):
    note(f"refused: {kind}")
    monkeypatch.setattr(sp, "_workspaces", {})
    call = CALLS[kind]()
    call()
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    refused = False
    try:
        with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=stream):
            call()
    except Exception as e:      # the refusal (ending an empty capture may raise on top of it)
        refused = any("workspace=" in str(x) for x in (e, e.__context__) if x is not None)
    assert refused
    torch.cuda.synchronize()
    want = call().clone()
    with torch.cuda.stream(stream):
        stream.wait_stream(torch.cuda.default_stream())
        got = call()
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_another_device_is_refused(monkeypatch):
    x = torch.ones(4, 64, dtype=torch.float16, device=DEV)
    A, B = torch.ones(2, 8, 64, dtype=torch.float16, device=DEV), torch.ones(2, 64, 8, dtype=torch.float16, device=DEV)
    cu, of = torch.arange(5, **I32), torch.zeros(4, **I32)
    lens, table = torch.ones(4, **I32), torch.zeros(4, 3, **I32)
    plan = sp.spear_adapter_plan(cu, of, 2, 4)
    y = torch.zeros_like(x)
    calls = {"block tables": lambda: sp.spear_kv_plan(lens, lens, lens, table, torch.zeros(9, **I32), torch.ones(1, **I32), 9),
             "plan": lambda: sp.spear_adapter_plan(cu, of, 2, 4), "adapters": lambda: sp.spear_adapter_add(y, x, A, B, plan),
             "draws": lambda: sp.spear_sample(x, torch.ones(4, 64, device=DEV))}
    for call in calls.values():
        call()
    torch.cuda.synchronize()
    y.zero_()
    with monkeypatch.context() as m:
        m.setattr(torch.cuda, "current_device", lambda: 1)
        for name, call in calls.items():
            note(f"another device: {name}")
            with pytest.raises(ValueError, match="current device is cuda:1"):
                call()
    torch.cuda.synchronize()
    assert not y.any()                          # nothing was launched


def test_two_streams_at_once():
    """The same calls on two streams, each with its own cached workspace."""
    note("two streams")
    calls = {n: make() for n, make in CALLS.items()}
    want = {n: call().clone() for n, call in calls.items()}
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(4):
        for name, call in calls.items():
            for s in streams:
                with torch.cuda.stream(s):
                    got.append((name, call()))
    torch.cuda.synchronize()
    for name, x in got:
        assert torch.equal(x, want[name]), name


# -------------------------------------------------------------- a serving step

class Server:
    """A one-layer model with adapters of its requests, and the state of its batch."""

    def __init__(self, rng, B, room, rows, pages, vocab=1000, hidden=256, heads=4, kv_heads=2, dim=64, adapters=3):
        self.B, self.rows, self.vocab, self.heads, self.kv_heads, self.dim = B, rows, vocab, heads, kv_heads, dim
        qkv = (heads + 2 * kv_heads) * dim
        self.linears, self.adapters = [], []
        for i, (K, N) in enumerate(((hidden, qkv), (heads * dim, hidden), (hidden, vocab))):
            _, W, EA, EB, w_g = workloads.random_layer(1, K, N, 16, seed=i)
            Wq, s = sp.spear_pack_w4(dev(W))
            self.linears.append((Wq, s, dev(EA), dev(EB), dev(w_g), 0.5))
            _, A, Bm, _ = ad.tensors(rng, 1, K, N, 16, adapters)
            self.adapters.append((dev(A), dev(Bm)))
        self.scale = dev(rng.normal(size=adapters).astype(np.float32))
        self.embed = dev(rng.normal(size=(vocab, hidden)).astype(np.float16))
        self.of = dev(rng.integers(-1, adapters, B).astype(np.int32))
        self.text = dev(rng.integers(0, vocab, (B, room + 1)))
        self.cache = sp.spear_kv_cache(pages, kv_heads, dim, 16, torch.float16, DEV)[:2]
        z = lambda *n: torch.zeros(*n, **I32)  # noqa: E731
        self.lens, self.ask, self.held, self.table = z(B), z(B), z(B), z(B, -(-room // 16))
        self.stack, self.count = dev(rng.permutation(pages).astype(np.int32)), torch.full((1,), pages, **I32)
        self.noise = torch.ones(B, vocab, device=DEV)
        self.rules = sa.settings([sa.RULES[b % len(sa.RULES)] for b in range(B)])
        self.ws = torch.zeros(64 << 20, dtype=torch.uint8, device=DEV)
        self.seen = {}

    def state(self):
        return [self.lens, self.ask, self.held, self.table, self.stack, self.count, self.text, *self.cache]

    def linear(self, i, x, plan):
        y = sp.spear_w4ec_linear(x, *self.linears[i], workspace=self.ws)
        base = y.clone()
        sp.spear_adapter_add(y, x, *self.adapters[i], plan, scale=self.scale, workspace=self.ws)
        self.seen[f"linear {i}"] = (x, base, y)
        return y

    def step(self):
        """New tokens of every sequence into the cache, and the token that follows where
        all of a sequence's are there: it becomes part of its text."""
        cu, _, slots, positions, sequence, _, _ = sp.spear_kv_plan(
            self.lens, self.ask, self.held, self.table, self.stack, self.count, self.rows, kv_lens=self.lens,
            held_out=self.held, free_out=self.count, workspace=self.ws)
        plan = sp.spear_adapter_plan(cu, self.of, len(self.scale), self.rows)
        x = self.embed[self.text[sequence.clamp(min=0).long(), positions.clamp(min=0).long()]]
        h, kv, d = self.heads, self.kv_heads, self.dim
        y = self.linear(0, x, plan)
        sp.spear_kv_append(y[:, h * d:(h + kv) * d].view(-1, kv, d), y[:, (h + kv) * d:].view(-1, kv, d), slots, *self.cache)
        o = torch.zeros(self.rows, h, d, dtype=torch.float16, device=DEV)
        sp.spear_paged_attention(y[:, :h * d].view(-1, h, d), *self.cache, self.table, cu, self.lens, self.rows, out=o,
                                 workspace=self.ws)
        x = self.linear(1, o.view(-1, h * d), plan)
        x = (x.float() * torch.rsqrt(x.float().pow(2).mean(-1, keepdim=True) + 1e-6)).half()
        z = self.linear(2, x, plan)
        n = cu[1:] - cu[:-1]
        last = torch.where(n > 0, cu[1:] - 1, -1).to(torch.int32)
        tokens, probs = sp.spear_sample(z, self.noise, rows=last, probs=True, workspace=self.ws, **self.rules)
        at = self.lens.long().clamp(max=self.text.shape[1] - 1)[:, None]
        self.text.scatter_(1, at, torch.where(n > 0, tokens, self.text.gather(1, at)[:, 0].int())[:, None].long())
        self.seen.update(cu=cu, slots=slots, positions=positions, sequence=sequence, logits=z, rows=last, tokens=tokens,
                         probs=probs)
        return [cu, slots, positions, sequence, tokens, probs]


def test_a_serving_step_eager_and_replayed():
    """Requests that start with prompts, go on by a token a step, end and start again,
    with fewer pages and rows than all of them ask for.  Every step: the plan as the
    oracle's, adapters and draws as the oracle's on what the GPU gave them, and a replay
    of the captured step gives the eager one's bits.  At the end the cache holds what
    one chunk over each sequence's text leaves there."""
    rng = np.random.default_rng(11)
    B, room, rows = 20, 150, 130
    s = Server(rng, B, room, rows, pages=70)
    s.ask.copy_(dev(rng.integers(0, 60, B).astype(np.int32)))
    first = [x.clone() for x in s.state()]
    s.step()                                    # (the products' first call)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        outs = s.step()
    for x, y in zip(s.state(), first):
        x.copy_(y)
    drawn = refused = 0
    for step in range(14):
        note(f"step {step}")
        s.noise.copy_(dev(rng.exponential(size=s.noise.shape).astype(np.float32)))
        before = [x.clone() for x in s.state()]
        eager = [x.clone() for x in s.step()]
        after = [x.clone() for x in s.state()]
        seen = {k: v for k, v in s.seen.items()}
        torch.cuda.synchronize()
        for x, y in zip(s.state(), before):
            x.copy_(y)
        g.replay()
        torch.cuda.synchronize()
        for x, y in zip((*outs, *s.state()), (*eager, *after)):
            assert torch.equal(x, y)
        n = lambda x: x.cpu().numpy()  # noqa: E731
        want = ref.kv_plan(*(n(x).astype(np.int64) for x in before[:3]), n(before[3]), n(before[4]), int(before[5]), rows, 16)
        got = [seen["cu"], s.lens, seen["slots"], seen["positions"], seen["sequence"], s.held, s.count, s.table, s.stack]
        for name, x, y in zip(kp.NAMES, got, want):
            assert np.array_equal(n(x), y), name
        cu, of = n(seen["cu"]), n(s.of)
        for i, (A, Bm) in enumerate(s.adapters):
            x, base, y = (n(v) for v in seen[f"linear {i}"])
            w, slack = ref.adapter_add(base, x, n(A), n(Bm), cu, of, n(s.scale))
            ad.compare(y, w, slack, base, cu, of, len(s.scale))
        z, tokens, probs = n(seen["logits"]), n(seen["tokens"]), n(seen["probs"])
        rules = {k: n(v) for k, v in s.rules.items()}
        served = np.diff(cu)
        for b in range(B):
            row = z[cu[b + 1] - 1] if served[b] > 0 else np.full(s.vocab, -np.inf, np.float16)
            rule = tuple(rules[k][b] for k in ("temperature", "top_k", "top_p", "min_p"))
            sa.check_row(b, row, n(s.noise[b]), rule, int(tokens[b]), probs[b])
        drawn += int((tokens >= 0).sum())
        refused += int(((n(before[1]) > 0) & (served == 0)).sum())
        # The next step's wishes: a token more, or the end and a new prompt.
        lens, ask = n(s.lens).copy(), n(before[1]).copy()
        ask[served > 0] = 1
        ask[(ask == 0) & (rng.random(B) < 0.5)] = 30
        gone = (rng.random(B) < 0.15) | (lens + ask > room)
        if step < 13:
            s.lens.copy_(dev(np.where(gone, 0, lens).astype(np.int32)))
            s.ask.copy_(dev(np.where(gone, 0, ask).astype(np.int32)))
    assert drawn > 100 and refused > 0
    for b in range(B):
        held = int(s.lens[b])
        if held == 0:
            continue
        x = s.embed[s.text[b, :held]]
        cu = torch.tensor([0, held], **I32)
        plan = sp.spear_adapter_plan(cu, s.of[b:b + 1], len(s.scale), held)
        y = sp.spear_w4ec_linear(x, *s.linears[0])
        sp.spear_adapter_add(y, x, *s.adapters[0], plan, scale=s.scale)
        at, kv, d = s.heads * s.dim, s.kv_heads, s.dim
        got = sp.spear_kv_gather(*s.cache, s.table[b:b + 1].contiguous(), cu, held)
        for i, x in enumerate(got):
            want = y[:, at + i * kv * d:at + (i + 1) * kv * d].view(-1, kv, d)
            # Linear layers of other row counts: fp16 results that may differ in their last
            # place (2^-11 of the value), before the adapter is added and rounded once more.
            tol = float(want.abs().max()) * 2 ** -10 + float(y.abs().max()) * 2 ** -11
            assert float((x.float() - want.float()).abs().max()) <= tol


def test_sampled_distributions_verify_their_own_drafts():
    """Drafts drawn from the distributions that verification then sees as both models':
    all are kept.  Against a target under other rules the kept ones are tokens that
    these rules leave."""
    note("drafts and their verification")
    rng = np.random.default_rng(12)
    B, K, V = 6, 4, 5000
    z = dev(sa.logits(rng, B * (K + 1), V))
    exp = lambda *n: dev(rng.exponential(size=n).astype(np.float32))  # noqa: E731
    rules = dict(temperature=0.8, top_k=50, top_p=0.9)
    at = torch.arange(B * (K + 1), **I32).view(B, K + 1)
    drafted, p_draft = [], []
    for k in range(K):
        tokens, p = sp.spear_sample(z, exp(B, V), rows=at[:, k].contiguous(), probs=True, **rules)
        drafted.append(tokens)
        p_draft.append(p)
    drafted, p_draft = torch.stack(drafted, 1), torch.stack(p_draft, 1)
    for b in range(B):
        for k in range(K):
            assert p_draft[b, k, drafted[b, k]] > 0
    _, target = sp.spear_sample(z, probs=True, **rules)
    assert torch.equal(target.view(B, K + 1, V)[:, :K], p_draft)
    u = dev(rng.random((B, K), dtype=np.float32))
    accepted, out = sp.spear_verify_draft(target.view(B, K + 1, V), p_draft, drafted, u, exp(B, V))
    assert accepted.tolist() == [K] * B and torch.equal(out[:, :K], drafted)
    assert (target.view(B, K + 1, V)[torch.arange(B), K, out[:, K].long()] > 0).all()
    _, target = sp.spear_sample(z, probs=True, temperature=1.0, top_k=5)
    accepted, out = sp.spear_verify_draft(target.view(B, K + 1, V), p_draft, drafted, u, exp(B, V))
    target = target.view(B, K + 1, V)
    for b in range(B):
        for k in range(int(accepted[b]) + 1):
            assert target[b, k, out[b, k]] > 0

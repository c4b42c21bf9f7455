"""The speculative decoding example: the W4 + EC linears, the paged cache, the
attention and the verification run together."""
import importlib.util
import os

import pytest
import torch

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "speculative_decoding.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("speculative_decoding", PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("dtype", [torch.int8, torch.float16])
def test_generation(example, dtype):
    """Lengths and tokens fit together, drafts are kept now and then, and what the
    cache holds after all rounds (chunks, single tokens, tokens taken back) is
    what one chunk over the same tokens leaves there."""
    print(f"[gpu-example] generate with {dtype}", flush=True)
    rounds, drafts, prompt, batch = 6, 3, 40, 3
    model, seqs, tokens, kept = example.generate(batch=batch, prompt=prompt, rounds=rounds, drafts=drafts, dtype=dtype,
                                                 seed=3)
    total = [prompt + sum(k[b] for k in kept) + rounds for b in range(batch)]
    assert [len(t) for t in tokens] == total
    assert all(0 <= x < model.vocab for t in tokens for x in t)
    assert all(0 <= k <= drafts for row in kept for k in row) and any(k > 0 for row in kept for k in row)
    assert seqs.lens.tolist() == [n - 1 for n in total]      # the last token is not cached yet
    import w4_gemm_gated_amd as sp
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    for b in range(batch):
        n = total[b] - 1
        again = example.Sequences(1, n + 1, model, g, dtype)
        again.lens += n
        text = torch.tensor(tokens[b][:n], device="cuda")
        model(text, again, example.offsets(n, 1), n, True)
        cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        want = sp.spear_kv_gather(again.cache[0], again.cache[1], again.table, cu, n, *again.cache[2:])
        got = sp.spear_kv_gather(seqs.cache[0], seqs.cache[1], seqs.table[b:b + 1].contiguous(), cu, n, *seqs.cache[2:])
        # Keys and values come from the embeddings alone, through linears of other
        # row counts: fp16 results that may differ in their last place (2^-11),
        # and codes by one step of 1/127 of the row's largest value there.
        for x, y in zip(got, want):
            tol = float(y.abs().max()) * (2 ** -10 if dtype is torch.float16 else 1 / 127 + 2 ** -10)
            assert float((x.float() - y.float()).abs().max()) <= tol

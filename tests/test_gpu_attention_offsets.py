"""Attention calls whose offsets do not rise: they end, within the tensors, and leave
the workspace's counters at zero; where the rows that such offsets repeat could pass
the kernels' 32-bit counts, nothing is computed."""
import numpy as np
import pytest
import torch

from oracle import spear_serve as ref
import w4_gemm_gated_amd as sp

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]
DEV = "cuda:0"


def note(msg):
    print(f"[gpu-offsets] {msg}", flush=True)


def inputs(batch, total, lens_most, group=1):
    g = torch.Generator(device=DEV)
    g.manual_seed(batch)
    q = torch.empty(total, group, 64, dtype=torch.float16, device=DEV).normal_(generator=g)
    k, v = (torch.empty(64, 1, 16, 64, dtype=torch.float16, device=DEV).normal_(generator=g) for _ in range(2))
    table = torch.randint(64, (batch, -(-lens_most // 16)), generator=g, device=DEV, dtype=torch.int32)
    lens = torch.randint(1, lens_most + 1, (batch,), generator=g, device=DEV, dtype=torch.int32)
    ws = torch.zeros(512 << 20, dtype=torch.uint8, device=DEV)
    out = torch.full((total, group, 64), 7.0, dtype=torch.float16, device=DEV)
    return q, k, v, table, lens, ws, out


# batch x rows / 16 x steps of 128 keys, and x rows / 128 x 64 keys: past 2^31 and 2^30
@pytest.mark.parametrize("batch,total,max_q,lens_most", [(65536, 262144, 1, 128), (65536, 131072, 1000, 1024)])
def test_large_calls_look_at_their_offsets(batch, total, max_q, lens_most):
    note(f"batch {batch}, {total} rows, max_q {max_q}")
    q, k, v, table, lens, ws, out = inputs(batch, total, lens_most)
    cu = torch.zeros(batch + 1, dtype=torch.int32, device=DEV)
    cu[1::2] = total
    sp.spear_paged_attention(q, k, v, table, cu, lens, max_q, out=out, workspace=ws)
    torch.cuda.synchronize()
    note("  offsets that fall: done")
    assert bool((out == 7).all()) and not ws[:1 << 20].any()
    # rising offsets of the same sizes: a few of the sequences against the oracle
    rng = np.random.default_rng(1)
    n = np.diff(np.concatenate([[0], np.sort(rng.integers(0, total + 1, size=batch - 1)), [total]]))
    cu = torch.from_numpy(np.concatenate([[0], np.cumsum(n)]).astype(np.int32)).to(DEV)
    sp.spear_paged_attention(q, k, v, table, cu, lens, max_q, out=out, workspace=ws)
    torch.cuda.synchronize()
    note("  rising offsets: done")
    assert not ws[:1 << 20].any()
    host = [x.cpu().numpy() for x in (q, k, v, table, cu, lens, out)]
    for b in [0, batch - 1, int(n.argmax())] + rng.integers(0, batch, size=12).tolist():
        at, end = int(host[4][b]), int(host[4][b + 1])
        want, spread, reach = ref.paged_attention(host[0][at:end], host[1], host[2], host[3][b:b + 1], [0, end - at],
                                                  host[5][b:b + 1], 0.125)
        # the bound of the attention tests, with this data's largest value
        tol = (2.0 ** -11 * np.abs(want) + (2.0 ** -11 + 2 * (2.0 ** -17 * reach[..., None] + 2.0 ** -18)) * spread
               + 2.0 ** -29 * 8 * lens_most + 2.0 ** -24)
        assert (np.abs(host[6][at:end].astype(np.float64) - want) <= tol).all()


@pytest.mark.parametrize("batch,total,max_q", [(300, 300, 1), (300, 900, 3), (90, 600, 600), (64, 4096, 64)])
def test_small_calls_with_falling_offsets_end(batch, total, max_q):
    note(f"batch {batch}, {total} rows, max_q {max_q}: offsets of all kinds")
    q, k, v, table, lens, ws, out = inputs(batch, total, 700, group=2)
    rng = np.random.default_rng(batch)
    for kind in ("zigzag", "falling", "wild"):
        cu = {"zigzag": np.where(np.arange(batch + 1) % 2, total, 0), "falling": np.linspace(total, 0, batch + 1),
              "wild": rng.integers(-2 ** 31, 2 ** 31, size=batch + 1)}[kind].astype(np.int32)
        sp.spear_paged_attention(q, k, v, table, torch.from_numpy(cu).to(DEV), lens, max_q, out=out, workspace=ws)
        torch.cuda.synchronize()
        note(f"  {kind}: done")
        assert not ws[:1 << 20].any()
        assert bool(torch.isfinite(out).all())

"""Attention tiles in which some waves compute nothing: a row tile's last waves
without rows, and (one query head to a kv head) first waves that see no key of the
diagonal's last tiles.  Their copies are the other waves' keys all the same."""
import numpy as np
import pytest
import torch

from test_gpu_paged_attention import check, make, note, run

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("q_lens,lens,kv_heads,group", [
    ([129], [4000], 2, 1),                       # one row in the last tile, 1 .. 4 key tiles of a row tile's own
    ([33], [4000], 2, 1), ([161], [2000], 1, 1),     # 33 rows: two waves idle
    ([96], [4000], 2, 1), ([224], [1500], 1, 1),     # 96: one
    ([43, 75], [3000, 2100], 1, 3),              # 129 and 225 rows of three heads
    ([400, 333], [400, 1000], 2, 1)])            # the diagonal: waves of a row tile end in different key tiles
def test_idle_waves(int8, dim, q_lens, lens, kv_heads, group):
    note(f"idle waves int8 {int8} dim {dim} q {q_lens} kv {lens} group {group}")
    c = make(np.random.default_rng(sum(lens) + dim), q_lens, lens, kv_heads, group, dim, 16, int8)
    got = run(c)
    check(c, got)
    for _ in range(3):
        assert np.array_equal(got.view(np.uint16), run(c).view(np.uint16))


@pytest.mark.parametrize("dim", [64, 128])
def test_idle_waves_on_a_full_gpu(dim):
    """As many row tiles with idle waves as fill the GPU, keys beyond the caches."""
    q_lens, lens = [33] * 24, [2500 + 37 * b for b in range(24)]
    note(f"idle waves, {len(lens)} sequences, dim {dim}")
    c = make(np.random.default_rng(dim), q_lens, lens, 8, 1, dim, 64, False)
    got = run(c)
    check(c, got)
    for _ in range(3):
        assert np.array_equal(got.view(np.uint16), run(c).view(np.uint16))

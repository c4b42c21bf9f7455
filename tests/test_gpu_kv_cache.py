"""The paged key/value cache on the GPU against the oracle: codes and scales bit
for bit, fp16 copies bit for bit, reading back, strides, padding, refusals."""
import numpy as np
import pytest
import torch

from oracle import spear_serve as ref
import w4_gemm_gated_amd as sp

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]
DEV = "cuda:0"


def note(msg):
    print(f"[gpu-kv-cache] {msg}", flush=True)


def rows_of(rng, n, heads, dim):
    """Keys as they come: ordinary rows, and rows of zeros, one value, tiny and
    huge values, ties, infinities and NaN."""
    x = rng.normal(size=(n, heads, dim)).astype(np.float16)
    special = [0.0, 65504.0, 6e-8, 2.5]
    for i in range(min(n // 3, len(special))):
        x[3 * i, 0] = special[i]
    if n > 20:
        x[13, -1, :4] = [127, 2.5, 3.5, -2.5]
        x[13, -1, 4:] = 0.5
        x[16, 0, 7] = np.inf
        x[17, 0, 9] = np.nan
    return x


def bits(a):
    return a.view({2: np.uint16, 4: np.uint32, 1: np.uint8}[a.dtype.itemsize])


@pytest.mark.parametrize("dtype", [torch.float16, torch.int8])
@pytest.mark.parametrize("heads,dim,page", [(1, 64, 16), (8, 128, 16), (3, 128, 64), (5, 64, 1024), (2, 128, 32)])
@pytest.mark.parametrize("tokens", [1, 7, 130])
def test_append_and_gather(dtype, heads, dim, page, tokens):
    note(f"append {dtype} heads {heads} dim {dim} page {page} tokens {tokens}")
    rng = np.random.default_rng(heads * 1000 + dim + page + tokens)
    pages = tokens // page + 4
    k, v = (rows_of(rng, tokens, heads, dim) for _ in range(2))
    # parts of a joint projection: token stride wider than the row, keys after values
    joint = torch.zeros(tokens, 3 * heads * dim + 8, dtype=torch.float16, device=DEV)
    kd = joint[:, 2 * heads * dim:3 * heads * dim].view(tokens, heads, dim)
    vd = joint[:, :heads * dim].view(tokens, heads, dim)
    kd.copy_(torch.from_numpy(k))
    vd.copy_(torch.from_numpy(v))
    slots = rng.permutation(pages * page)[:tokens].astype(np.int64)
    slots[tokens // 2] = -1
    if tokens > 6:
        slots[3] = pages * page + 5             # outside: not written
    kc, vc, ks, vs = sp.spear_kv_cache(pages, heads, dim, page, dtype, DEV)
    kc.fill_(3)
    vc.fill_(5)
    want = {n: (c.cpu().numpy().copy(), s.cpu().numpy().copy() if s is not None else None)
            for n, c, s in (("k", kc, ks), ("v", vc, vs))}
    sp.spear_kv_append(kd, vd, torch.from_numpy(slots).to(DEV), kc, vc, ks, vs)
    torch.cuda.synchronize()
    for x, n in ((k, "k"), (v, "v")):
        cache, scale = want[n]
        codes, s = ref.quantise_kv(x)
        for i, slot in enumerate(slots):
            if not 0 <= slot < pages * page:
                continue
            cache[slot // page, :, slot % page] = codes[i] if dtype is torch.int8 else x[i]
            if scale is not None:
                scale[slot // page, :, slot % page] = s[i]
    for c, s, n in ((kc, ks, "k"), (vc, vs, "v")):
        assert np.array_equal(bits(c.cpu().numpy()), bits(want[n][0])), n
        if s is not None:
            got, exp = s.cpu().numpy(), want[n][1]
            assert np.array_equal(np.isnan(got), np.isnan(exp))
            assert np.array_equal(bits(got[~np.isnan(exp)]), bits(exp[~np.isnan(exp)]))


@pytest.mark.parametrize("dtype", [torch.float16, torch.int8])
@pytest.mark.parametrize("lens", [[1], [0, 17, 0, 0, 33, 1, 64], [200, 3, 129], [0, 0], [1] * 150 + [0] * 70 + [5] * 9])
@pytest.mark.parametrize("heads,dim,page", [(8, 128, 16), (3, 64, 32)])
def test_gather_ragged(dtype, lens, heads, dim, page):
    note(f"gather {dtype} lens {lens[:7]} heads {heads} dim {dim} page {page}")
    rng = np.random.default_rng(len(lens) + dim)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 2
    order = rng.permutation(pages)
    table = np.full((len(lens), max(need) + 1), -1, dtype=np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    if dtype is torch.int8:
        caches = [rng.integers(-127, 128, size=(pages, heads, page, dim)).astype(np.int8) for _ in range(2)]
        scales = [rng.lognormal(-4, 2, size=(pages, heads, page)).astype(np.float32) for _ in range(2)]
    else:
        caches = [rng.normal(size=(pages, heads, page, dim)).astype(np.float16) for _ in range(2)]
        scales = [None, None]
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    extra = 5
    d = lambda a: None if a is None else torch.from_numpy(a).to(DEV)  # noqa: E731
    got = sp.spear_kv_gather(d(caches[0]), d(caches[1]), d(table), d(cu), int(cu[-1]) + extra, d(scales[0]),
                             d(scales[1]))
    torch.cuda.synchronize()
    for x, c, s in zip(got, caches, scales):
        x = x.cpu().numpy()
        assert not x[cu[-1]:].any()
        for b, n in enumerate(lens):
            for i in range(n):
                p, o = table[b, i // page], i % page
                if s is None:
                    want = c[p, :, o]
                else:
                    with np.errstate(over="ignore"):
                        want = (c[p, :, o].astype(np.float32) * s[p, :, o][:, None]).astype(np.float16)
                assert np.array_equal(bits(x[cu[b] + i]), bits(want)), (b, i)


@pytest.mark.parametrize("dtype", [torch.float16, torch.int8])
@pytest.mark.parametrize("heads,dim,page", [(9, 128, 16), (17, 64, 64)])
def test_large_outputs(dtype, heads, dim, page):
    """Outputs past 256 MiB (a thread takes two rows there): many sequences of odd
    lengths, some empty, and rows of no sequence at the end; the same bits as the
    definition in fp32 torch operations, row by row."""
    rng = np.random.default_rng(dim + heads)
    lens = rng.integers(0, 1400, size=90).tolist()
    lens[4] = lens[5] = lens[89] = 0
    total, rows = sum(lens), sum(lens) + 37
    rows += max(0, (1 << 28) // (heads * dim * 4) + 3 - rows)
    note(f"large gather {dtype} heads {heads} dim {dim} rows {rows} of which {total} cached")
    g = torch.Generator(device=DEV)
    g.manual_seed(dim)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + 1
    order = torch.randperm(pages, generator=g, device=DEV)
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n].int()
        at += n
    shape = (pages, heads, page, dim)
    if dtype is torch.int8:
        caches = [torch.randint(-127, 128, shape, generator=g, device=DEV).to(torch.int8) for _ in range(2)]
        scales = [torch.rand(shape[:3], generator=g, device=DEV) for _ in range(2)]
    else:
        caches = [torch.randn(shape, generator=g, device=DEV).half() for _ in range(2)]
        scales = [None, None]
    cu = torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device=DEV)
    out = sp.spear_kv_gather(*caches, table, cu, rows, k_scale=scales[0], v_scale=scales[1])
    row = torch.arange(total, device=DEV)
    b = torch.bucketize(row, cu[1:].long(), right=True)
    i = row - cu.long()[b]
    place = table[b, i // page].long()
    for got, cache, scale in zip(out, caches, scales):
        assert torch.count_nonzero(got[total:]).item() == 0
        for r in range(0, total, 16384):
            p, o = place[r:r + 16384], (i % page)[r:r + 16384]
            want = cache[p, :, o]
            if scale is not None:
                want = (want.float() * scale[p, :, o][..., None]).half()
            assert torch.equal(got[r:r + 16384][:want.shape[0]], want)


def test_offsets_past_32_bits():
    """A cache of more than 2^32 bytes (and 2^31 values): its last pages are
    written and read back."""
    heads, dim, page = 8, 128, 64
    pages = (1 << 31) // (heads * dim * page) + 4
    for dtype in (torch.float16, torch.int8):
        note(f"large cache {dtype} pages {pages}")
        kc, vc = (torch.empty(pages, heads, page, dim, dtype=dtype, device=DEV) for _ in range(2))
        ks, vs = ((torch.empty(pages, heads, page, device=DEV) for _ in range(2)) if dtype is torch.int8
                  else (None, None))
        x = torch.randn(3, heads, dim, device=DEV).half()
        slots = torch.tensor([pages * page - 1, (pages - 2) * page, 5], device=DEV)
        sp.spear_kv_append(x, -x, slots, kc, vc, ks, vs)
        table = torch.tensor([[pages - 2]], dtype=torch.int32, device=DEV)
        k, v = sp.spear_kv_gather(kc, vc, table, torch.tensor([0, 1], dtype=torch.int32, device=DEV), 1, ks, vs)
        tol = 0 if dtype is torch.float16 else float(x[1].abs().max()) / 127 * 0.51 + 2 ** -10
        assert float((k[0] - x[1]).abs().max()) <= tol and float((v[0] + x[1]).abs().max()) <= tol
        last = kc[pages - 1, :, page - 1].float() * (1 if ks is None else ks[pages - 1, :, page - 1, None])
        assert float((last - x[0].float()).abs().max()) <= (tol or 0) + 0.02 * (dtype is torch.int8)
        del kc, vc, ks, vs


def test_other_stream_and_out_arguments():
    note("gather on another stream")
    kc, vc, _, _ = sp.spear_kv_cache(4, 2, 64, 16, torch.float16, DEV)
    x = torch.randn(20, 2, 64, device=DEV).half()
    slots = torch.arange(20, device=DEV)
    table = torch.arange(2, dtype=torch.int32, device=DEV)[None].contiguous()
    cu = torch.tensor([0, 20], dtype=torch.int32, device=DEV)
    ko, vo = torch.empty_like(x), torch.empty_like(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        sp.spear_kv_append(x, x, slots, kc, vc)
        got = sp.spear_kv_gather(kc, vc, table, cu, 20, k_out=ko, v_out=vo)
    s.synchronize()
    assert got[0] is ko and torch.equal(ko, x) and torch.equal(vo, x)
    sp.spear_kv_append(x[:0], x[:0], slots[:0], kc, vc)       # nothing to write
    assert sp.spear_kv_gather(kc, vc, table, cu, 0)[0].shape == (0, 2, 64)


def test_refusals():
    kc, vc, ks, vs = sp.spear_kv_cache(4, 2, 64, 16, torch.int8, DEV)
    x = torch.zeros(3, 2, 64, dtype=torch.float16, device=DEV)
    slots = torch.zeros(3, dtype=torch.int64, device=DEV)
    with pytest.raises(ValueError):
        sp.spear_kv_append(x, x, slots, kc, vc)                       # no scales
    with pytest.raises(TypeError):
        sp.spear_kv_append(x, x, slots.int(), kc, vc, ks, vs)
    with pytest.raises(TypeError):
        sp.spear_kv_append(x.float(), x, slots, kc, vc, ks, vs)
    with pytest.raises(ValueError):
        sp.spear_kv_append(x, x[:2], slots, kc, vc, ks, vs)
    with pytest.raises(ValueError):
        sp.spear_kv_append(x.transpose(1, 2), x, slots, kc, vc, ks, vs)
    with pytest.raises(ValueError):
        sp.spear_kv_append(x, x, slots.cpu(), kc, vc, ks, vs)
    odd = torch.zeros(3, 2 * 64 + 4, dtype=torch.float16, device=DEV)[:, :128].view(3, 2, 64)
    with pytest.raises(sp.SpearError, match="INVALID_SHAPE"):
        sp.spear_kv_append(odd, odd, slots, kc, vc, ks, vs)           # stride not a multiple of 8
    for dim, page in ((96, 16), (64, 8), (64, 48), (64, 2048)):
        c = [torch.zeros(2, 2, page, dim, dtype=torch.float16, device=DEV) for _ in range(2)]
        y = torch.zeros(3, 2, dim, dtype=torch.float16, device=DEV)
        with pytest.raises(sp.SpearError, match="UNSUPPORTED"):
            sp.spear_kv_append(y, y, slots, *c)
    cu = torch.tensor([0, 3], dtype=torch.int32, device=DEV)
    table = torch.zeros(1, 1, dtype=torch.int32, device=DEV)
    with pytest.raises(ValueError):
        sp.spear_kv_gather(kc, vc, table, cu[:1], 3, ks, vs)
    with pytest.raises(sp.SpearError, match="INVALID_SHAPE"):
        sp.spear_kv_gather(kc, vc, table[:, :0].contiguous(), cu, 3, ks, vs)


@pytest.mark.parametrize("dtype", [torch.float16, torch.int8])
@pytest.mark.parametrize("cu", [[5, 9, 0], [100, 60, 50], [2 ** 31 - 1, 3, 40], [-2 ** 31, -2 ** 31, 2 ** 31 - 1],
                                [0, 40, 7], [0, -9, 30], [70, 70, 70]])
def test_offsets_that_do_not_rise_stay_inside(dtype, cu):
    """Rows that the offsets place before a sequence's first are zero; every other
    row holds some token of the cache: nothing outside the tensors is read."""
    note(f"gather {dtype} offsets {cu}")
    heads, dim, page, rows, batch = 2, 64, 16, 64, len(cu) - 1
    kc, vc, ks, vs = sp.spear_kv_cache(5, heads, dim, page, dtype, DEV)
    for x, a in ((kc, 1), (vc, 2)):
        x.fill_(a)                              # every place of the cache holds this
    for x in (ks, vs):
        if x is not None:
            x.fill_(1.0)
    # the table in the middle of a larger one, whose other entries name a page of other values
    kc[4] = vc[4] = 99
    wide = torch.full((batch + 6, 3), 4, dtype=torch.int32, device=DEV)
    wide[3:3 + batch] = torch.arange(3 * batch, dtype=torch.int32, device=DEV).view(batch, 3) % 4
    k, v = sp.spear_kv_gather(kc, vc, wide[3:3 + batch], torch.tensor(cu, dtype=torch.int32, device=DEV), rows, ks, vs)
    torch.cuda.synchronize()
    for x, a in ((k, 1), (v, 2)):
        assert bool(((x == 0) | (x == a)).all())
        assert bool((x.flatten(1) == x[:, :1, 0]).all())            # whole rows
    if cu[0] > 0 and cu[1] > 0:                 # no row before the smallest offset belongs to a sequence
        assert not k[:min(max(min(cu), 0), rows)].any()


@pytest.mark.parametrize("dtype", [torch.float16, torch.int8])
@pytest.mark.parametrize("pages", [0, 3])
def test_gather_of_no_sequences_gives_zeros(dtype, pages):
    note(f"gather of no sequences {dtype}")
    kc, vc, ks, vs = sp.spear_kv_cache(2, 3, 64, 16, dtype, DEV)
    out = [torch.full((70, 3, 64), 9.0, dtype=torch.float16, device=DEV) for _ in range(2)]
    table = torch.zeros(0, pages, dtype=torch.int32, device=DEV)
    sp.spear_kv_gather(kc, vc, table, torch.zeros(1, dtype=torch.int32, device=DEV), 70, ks, vs, *out)
    torch.cuda.synchronize()
    assert not out[0].any() and not out[1].any()

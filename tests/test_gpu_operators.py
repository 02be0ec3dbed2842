"""Operators on a caller's own buffers against their definitions in float64:
attention of chunks over a paged cache, eviction by accumulated weight, and
the logits rules; alone, captured into graphs, and run together."""
import math

import numpy as np
import pytest
import torch

from operator_common import AttnCase, close, evict_rule, rules_rule

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def R():
    import __graft_entry__ as g
    g.build()
    from speculative_whisper_asr_gb300 import runtime
    return runtime


# ------------------------------------------------------------------ attention
def _attend(R, c, mass=True, lse=True, cache=None, **kw):
    cache = cache or R.PagedCache(c.k, c.v, c.table)
    out = torch.full_like(c.q, 7.0)
    ls = torch.full(c.q.shape[:2], 7.0, device="cuda") if lse else None
    ms = c.mass0.clone() if mass else None
    cache.attend(c.q, c.kv_len, c.cu, max_q=c.max_q, max_kv=c.max_kv, causal=c.causal, scale=c.scale, out=out, lse=ls,
                 mass=ms, req_ids=c.req, **kw)
    torch.cuda.synchronize()
    return out, ls, ms


def _check(R, c, bad_pages=(), **kw):
    out, lse, mass = _attend(R, c, **kw)
    want, tol = c.reference(bad_pages)
    n = c.rows
    close("out", out[:n], want[0], tol[0])
    assert bool((out[n:] == 7.0).all())                       # rows outside every chunk are left as they were
    if lse is not None:
        close("lse", lse[:n], want[1], tol[1])
        assert bool((lse[n:] == 7.0).all())
    if mass is not None:
        close("mass", mass, want[2], tol[2])
        for s, L in enumerate(c.slot_len):                    # behind the cache: untouched
            assert torch.equal(mass[s, :, L:], c.mass0[s, :, L:])
    return out, lse, mass


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("chunks,lens", [
    ([1], [1]), ([1], [448]), ([9, 4, 1], [64, 65, 63]), ([2, 0, 5], [31, 100, 0]), ([16, 9], [33, 130]),
    ([17, 33], [200, 129]), ([100, 129], [100, 300]), ([40], [1000]), ([300, 1], [700, 513]),
    ([12, 3], [5, 2]),                                        # chunks longer than their cache: rows that see nothing
])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_matches_definition(R, dtype, chunks, lens, causal):
    _check(R, AttnCase(chunks, lens, dtype=dtype, causal=causal, seed=len(lens) + sum(chunks)))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("page", [1, 7, 8, 16, 32, 64, 100, 128, 200])
@pytest.mark.parametrize("layout", ["head", "token"])
def test_attention_page_sizes_and_layouts(R, dtype, page, layout):
    _check(R, AttnCase([3, 20, 50], [190, 201, 130], page=page, dtype=dtype, layout=layout, seed=page))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (6, 1), (8, 8), (8, 2), (5, 5), (32, 2), (40, 1)])
@pytest.mark.parametrize("chunks", [[1, 1], [9, 2], [70, 31]])
def test_attention_head_layouts(R, dtype, hq, hkv, chunks):
    _check(R, AttnCase(chunks, [150, 97], hq=hq, hkv=hkv, dtype=dtype, seed=hq))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("chunks,lens", [([1, 1], [150, 97]), ([3, 2], [70, 33])])
def test_attention_many_heads_share_one(R, dtype, chunks, lens):
    """More query heads per KV head than a row tile holds."""
    _check(R, AttnCase(chunks, lens, hq=140, hkv=1, dtype=dtype, seed=140))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("c", [1, 2, 3, 8, 9, 16, 17, 32, 33])
@pytest.mark.parametrize("kv", [63, 64, 65, 1025])
def test_attention_around_the_row_tiles(R, dtype, c, kv):
    _check(R, AttnCase([c], [kv], hq=2, hkv=2, dtype=dtype, seed=c + kv))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("chunks", [[2, 1, 3], [64, 40, 33]])
def test_attention_slots_and_bad_ids(R, dtype, chunks):
    c = AttnCase(chunks, [70, 90, 11], dtype=dtype, req_ids=[4, -1, 1], slots=6, seed=3)
    _check(R, c)
    c = AttnCase(chunks, [70, 90, 11], dtype=dtype, req_ids=[5, 0, 6], slots=6, seed=4)
    _check(R, c)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("chunks", [[5], [80]])
@pytest.mark.parametrize("page", [16, 64, 100])
def test_attention_skips_bad_pages(R, dtype, chunks, page):
    c = AttnCase(chunks, [330], dtype=dtype, page=page, causal=False, seed=page)
    c.table[0, 1] = -3
    c.table[0, 3] = c.k.shape[0]
    _check(R, c, bad_pages=(1, 3))
    one = AttnCase(chunks, [page], dtype=dtype, page=page, causal=False, seed=page)
    one.table[0, 0] = one.k.shape[0] + 5
    _check(R, one, bad_pages=(0,))                            # nothing left to see


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("chunks", [[7], [90]])
def test_attention_optional_outputs_and_strides(R, dtype, chunks):
    c = AttnCase(chunks, [140], hq=4, hkv=4, dtype=dtype, seed=9)
    wide = torch.randn(c.q.shape[0], 12, 64, device="cuda").to(dtype)      # q inside a fused q|k|v row
    wide[:, 4:8] = c.q
    c.q = wide[:, 4:8]
    want, tol = c.reference()
    cache = R.PagedCache(c.k, c.v, c.table)
    big = torch.full((c.q.shape[0], 7, 64), 7.0, device="cuda", dtype=dtype)
    out = big[:, 2:6]
    for mass in (None, c.mass0.clone()):
        cache.attend(c.q, c.kv_len, c.cu, max_q=c.max_q, max_kv=c.max_kv, out=out, mass=mass)
        torch.cuda.synchronize()
        close("out", out[: c.rows], want[0], tol[0])
        assert bool((big[:, :2] == 7.0).all()) and bool((big[:, 6:] == 7.0).all())
        if mass is not None:
            close("mass", mass, want[2], tol[2])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("amp", [0.0, 12.0])
@pytest.mark.parametrize("scale", [0.125, -0.3, 0.0])
def test_attention_score_ranges(R, dtype, amp, scale):
    """All scores equal, one score far above the rest, a negative scale."""
    _check(R, AttnCase([9, 70], [300, 301], dtype=dtype, amp=amp, scale=scale, seed=11))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("chunks,lens", [([1], [5000]), ([1, 1], [4097, 300]), ([9], [3000]), ([130], [2500])])
def test_attention_long_caches(R, dtype, chunks, lens):
    _check(R, AttnCase(chunks, lens, hq=4, hkv=2, dtype=dtype, seed=sum(lens)))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("chunks", [[3, 5], [66, 20]])
def test_attention_growing_maximum(R, dtype, chunks):
    """Keys that grow along the cache: the running maximum moves at every tile."""
    c = AttnCase(chunks, [400, 333], hq=2, hkv=2, dtype=dtype, causal=False, seed=2)
    for s, L in enumerate(c.slot_len):
        for j in range(L):
            c.k[c.table[s, j // 64], :, j % 64] *= 0.02 * j
    _check(R, c)


def test_attention_host_bounds_cut(R):
    """max_q and max_kv below the device lengths: nothing is read or written behind them."""
    c = AttnCase([8], [200], causal=False, seed=1)
    want, tol = AttnCase([8], [200], causal=False, seed=1).reference()
    cache = R.PagedCache(c.k, c.v, c.table)
    out = torch.full_like(c.q, 7.0)
    cache.attend(c.q, c.kv_len, c.cu, max_q=5, max_kv=200, causal=False, out=out)
    torch.cuda.synchronize()
    close("out", out[:5], want[0][:5], tol[0][:5])
    assert bool((out[5:] == 7.0).all())
    short = AttnCase([8], [200], causal=False, seed=1)
    short.slot_len, short.lens = [130], [130]
    want, tol = short.reference()
    mass = c.mass0.clone()
    cache.attend(c.q, c.kv_len, c.cu, max_q=8, max_kv=130, causal=False, out=out, mass=mass)
    torch.cuda.synchronize()
    close("out", out[:8], want[0], tol[0])
    close("mass", mass, want[2], tol[2])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("chunks,lens", [([9, 3], [448, 300]), ([1], [4000]), ([150, 64], [600, 64])])
def test_attention_same_bits_twice_and_in_a_graph(R, dtype, chunks, lens):
    c = AttnCase(chunks, lens, dtype=dtype, seed=6)
    cache = R.PagedCache(c.k, c.v, c.table)
    a, b = _attend(R, c, cache=cache), _attend(R, c, cache=cache)
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    # captured: the lengths are read at replay
    out, lse, mass = torch.zeros_like(c.q), torch.zeros(c.q.shape[:2], device="cuda"), c.mass0.clone()
    lens_dev, full = torch.zeros_like(c.kv_len), c.kv_len
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.attend(c.q, lens_dev, c.cu, max_q=c.max_q, max_kv=c.max_kv, out=out, lse=lse, mass=mass)
    big = AttnCase([c.max_q + 60], [c.max_kv + 900], hq=8, hkv=2, dtype=dtype)     # a larger eager call in between
    cache2 = R.PagedCache(big.k, big.v, big.table)
    _attend(R, big, cache=cache2)
    lens_dev.copy_(full)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out[: c.rows], a[0][: c.rows]) and torch.equal(lse[: c.rows], a[1][: c.rows])
    assert torch.equal(mass, a[2])
    lens_dev.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert bool((out[: c.rows] == 0).all()) and bool((lse[: c.rows] == -math.inf).all()) and torch.equal(mass, a[2])


def test_attention_two_streams(R):
    c, d = AttnCase([9] * 4, [448, 300, 20, 128], seed=1), AttnCase([64] * 3, [900, 700, 64], seed=2)
    want = [_attend(R, x) for x in (c, d)]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    torch.cuda.synchronize()
    for x, s in ((c, s1), (d, s2)):
        with torch.cuda.stream(s):
            out, lse, mass = torch.full_like(x.q, 7.0), torch.full(x.q.shape[:2], 7.0, device="cuda"), x.mass0.clone()
            R.PagedCache(x.k, x.v, x.table).attend(x.q, x.kv_len, x.cu, max_q=x.max_q, max_kv=x.max_kv, out=out,
                                                   lse=lse, mass=mass)
            got.append((out, lse, mass))
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        for x, y in zip(a, b):
            assert torch.equal(x, y)


def test_attention_offsets_past_32_bits(R):
    """A page whose elements lie more than 2^32 elements into the pool."""
    page, heads = 64, 1
    stride = 1 << 20                                          # elements between pages
    pages = 4200
    flat = torch.empty(pages * stride + 64 * 64, dtype=BF, device="cuda")
    k = torch.as_strided(flat, (pages, heads, page, 64), (stride, 64 * 64, 64, 1))
    v = torch.as_strided(flat, (pages, heads, page, 64), (stride, 64 * 64, 64, 1), 64 * 64)
    c = AttnCase([5], [130], hq=2, hkv=1, seed=8)
    far = torch.tensor([4198, 3, 4100], device="cuda")
    k[far] = c.k[c.table[0, :3].long()]
    v[far] = c.v[c.table[0, :3].long()]
    c.k, c.v = k, v
    want, tol = None, None
    kk, vv, table = c.k, c.v, far.to(torch.int32)[None].contiguous()
    near = AttnCase([5], [130], hq=2, hkv=1, seed=8)
    want, tol = near.reference()
    out = torch.zeros_like(c.q)
    cache = R.PagedCache(kk, vv, table)
    mass = c.mass0.clone()
    cache.attend(c.q, c.kv_len, c.cu, max_q=5, max_kv=130, out=out, mass=mass)
    torch.cuda.synchronize()
    close("out", out[:5], want[0], tol[0])
    close("mass", mass, want[2], tol[2])
    # and an eviction moves rows between such places
    before = kk[far, 0].reshape(-1, 64)[:130].clone()
    kept = evict_rule(mass[0, 0].cpu(), 130, 70, 1, 5)
    lens = c.kv_len.clone()
    cache.evict(lens, mass, keep=70, max_kv=130, sink=1, recent=5)
    torch.cuda.synchronize()
    assert torch.equal(kk[far[:2], 0].reshape(-1, 64)[:70], before[kept])


def test_wrong_tensors_raise(R):
    c = AttnCase([2], [10], seed=1)
    cache = R.PagedCache(c.k, c.v, c.table)
    args = dict(max_q=2, max_kv=10)
    for bad in (dict(q=c.q.float()), dict(kv_len=c.kv_len.long()), dict(cu_q=c.cu.cpu()),
                dict(q=c.q.transpose(0, 1)), dict(lse=torch.zeros(1, 1, device="cuda")),
                dict(mass=torch.zeros(1, 1, 10, device="cuda")), dict(mass=torch.zeros(1, 2, 5, device="cuda"))):
        a = dict(q=c.q, kv_len=c.kv_len, cu_q=c.cu, **args)
        a.update(bad)
        with pytest.raises((ValueError, R.B.WSError)):
            cache.attend(**a)
    with pytest.raises(ValueError):
        R.PagedCache(c.k, c.v.float(), c.table)
    with pytest.raises(ValueError):
        R.PagedCache(c.k, c.v, c.table.long())


@pytest.mark.parametrize("c,G", [(33, 1), (40, 1), (41, 1), (48, 1), (10, 4), (11, 4), (5, 8), (6, 7)])
@pytest.mark.parametrize("causal", [True, False])
def test_attention_between_streaming_and_wide_row_tiles(R, c, G, causal):
    """33 to 48 rows per KV head: two streaming row tiles, or one of 128 rows."""
    _check(R, AttnCase([c, 3, c], [600, 64, 37], hq=2 * G, hkv=2, causal=causal, seed=c * G))
    _check(R, AttnCase([c], [1700], hq=2 * G, hkv=2, causal=causal, seed=c + G))


@pytest.mark.parametrize("c,kv", [(1, 4096), (1, 4097), (8, 4096), (9, 2048), (9, 2049), (16, 2048), (32, 2048), (32, 2049)])
@pytest.mark.parametrize("page", [64, 100])
def test_attention_scores_that_just_fit(R, c, kv, page):
    """Weights with the longest caches whose scores one CTA keeps, and one position more."""
    _check(R, AttnCase([c] * 10, [kv, 1, 700] + [40] * 7, hq=8, hkv=8, page=page, causal=c < 32, seed=c + kv))


@pytest.mark.parametrize("c", [15, 16, 17, 31, 32, 33, 47])
@pytest.mark.parametrize("n", [2, 40])
def test_fp32_row_tiles(R, c, n):
    """Around the fp32 row tiles of 16, 32 and 64 rows, with few requests (joined key ranges) and many."""
    lens = [max(c, 30 + 53 * (i % 7)) for i in range(n)]
    _check(R, AttnCase([c if i % 3 else max(1, c - 9) for i in range(n)], lens, dtype=F32, seed=c + n))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("c", [1, 6, 30, 90])
def test_attention_nan_row_stays_alone(R, dtype, c):
    """A NaN in one query row makes that row NaN and no other."""
    x = AttnCase([c, c], [300, 130], dtype=dtype, hq=4, hkv=2, seed=c)
    want, tol = x.reference()
    x.q[c - 1, 2, 5] = math.nan
    out, lse, _ = _attend(R, x, mass=False)
    assert bool(out[c - 1, 2].isnan().all()) and bool(lse[c - 1, 2].isnan())
    for got, w, t in ((out, want[0], tol[0]), (lse, want[1], tol[1])):
        got = got[: 2 * c].double().cpu()
        got[c - 1, 2] = w[c - 1, 2]
        close("rows beside a NaN row", got, w, t)


def test_a_refused_call_leaves_the_next_one_alone(R):
    """Sizes of a refused call are not remembered: the same sizes with sound arguments go through."""
    c = AttnCase([90], [300], seed=4)
    cache = R.PagedCache(c.k, c.v, c.table)
    with pytest.raises(R.B.WSError):
        cache.attend(c.q, c.kv_len, c.cu, max_q=c.max_q, max_kv=c.max_kv, causal=c.causal, scale=c.scale,
                     mass=c.mass0[:, :, :5].contiguous())
    out, lse, mass = _attend(R, c, lse=False, cache=cache)
    want, tol = c.reference()
    close("out", out[: c.rows], want[0], tol[0])
    close("mass", mass, want[2], tol[2])
    m, n = mass.clone(), int(c.kv_len[0])
    with pytest.raises(R.B.WSError):
        cache.evict(c.kv_len, m, keep=100, max_kv=n, mass_out=m[:, :, :20].contiguous())
    kept = evict_rule(mass[0, 0].cpu().numpy(), n, 100, 0, 0)
    cache.evict(c.kv_len, m, keep=100, max_kv=n)
    torch.cuda.synchronize()
    assert int(c.kv_len[0]) == 100 and torch.equal(m[0, 0, :100], mass[0, 0, kept])


def test_strided_page_table_is_refused(R):
    """Rows of a wider table: the entries behind the last row's may not exist."""
    c = AttnCase([2], [200], seed=1)
    wide = torch.zeros(3, 9, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        R.PagedCache(c.k, c.v, wide[:, 4:])


# ------------------------------------------------------------------ eviction
def _evict_case(R, lens, page, dtype, keep, sink, recent, hkv=3, layout="head", in_place=False, seed=0, odd=False):
    g = torch.Generator(device="cpu").manual_seed(seed)
    n, width = len(lens), max(1, max(-(-x // page) for x in lens))
    out_w = -(-keep // page)
    pages = n * (width + out_w) + 1
    shape = (pages, hkv, page, 64) if layout == "head" else (pages, page, hkv, 64)
    k, v = (torch.randn(shape, generator=g).to(dtype).cuda() for _ in range(2))
    if layout != "head":
        k, v = k.permute(0, 2, 1, 3), v.permute(0, 2, 1, 3)
    perm = torch.randperm(pages, generator=g)
    table = perm[: n * width].reshape(n, width).to(torch.int32).cuda()
    tout = None if in_place else perm[n * width: n * (width + out_w)].reshape(n, out_w).to(torch.int32).cuda()
    M = max(keep, max(lens)) + 3
    mass = torch.rand(n, hkv, M, generator=g)
    mass = torch.where(torch.rand(mass.shape, generator=g) < 0.3, (mass * 4).round() / 4, mass)    # ties
    if odd:
        r = torch.rand(mass.shape, generator=g)
        mass = torch.where(r < 0.05, torch.full_like(mass, math.nan), mass)
        mass = torch.where((r > 0.05) & (r < 0.1), -mass, mass)
        mass = torch.where((r > 0.1) & (r < 0.12), torch.full_like(mass, math.inf), mass)
        mass = torch.where((r > 0.12) & (r < 0.2), torch.full_like(mass, -0.0), mass)
    mass = mass.cuda()
    pos = torch.randint(0, 1 << 30, mass.shape, generator=g, dtype=torch.int32).cuda()
    kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
    k0, v0, m0, p0 = k.clone(), v.clone(), mass.clone(), pos.clone()
    cache = R.PagedCache(k, v, table)
    if in_place:
        cache.evict(kv_len, mass, keep=keep, max_kv=max(keep, max(lens)), sink=sink, recent=recent, pos=pos)
        new_len, m1, p1, dst = kv_len, mass, pos, table
    else:
        new_len = torch.full_like(kv_len, -5)
        m1 = torch.full((n, hkv, keep + 2), 5.0, device="cuda")
        p1 = torch.full((n, hkv, keep + 1), 5, dtype=torch.int32, device="cuda")
        cache.evict(kv_len, mass, keep=keep, max_kv=max(keep, max(lens)), sink=sink, recent=recent, page_table_out=tout,
                    kv_len_out=new_len, mass_out=m1, pos=pos, pos_out=p1)
        dst = tout
        assert kv_len.tolist() == list(lens) and torch.equal(mass.view(torch.int32), m0.view(torch.int32))
    torch.cuda.synchronize()
    assert new_len.tolist() == [min(x, keep) for x in lens]
    # what the pool, the masses and the labels have to hold, everything else untouched
    wk, wv = k0.clone(), v0.clone()
    wm = m0.clone() if in_place else torch.full_like(m1, 5.0)
    wp = p0.clone() if in_place else torch.full_like(p1, 5)
    for s, L in enumerate(lens):
        for h in range(hkv):
            kept = torch.tensor(evict_rule(m0[s, h].cpu().numpy(), L, keep, sink, recent), dtype=torch.long, device="cuda")
            j = torch.arange(len(kept), device="cuda")
            a, b = table[s].long(), dst[s].long()
            wk[b[j // page], h, j % page] = k0[a[kept // page], h, kept % page]
            wv[b[j // page], h, j % page] = v0[a[kept // page], h, kept % page]
            wm[s, h, : len(kept)] = m0[s, h, kept]
            wp[s, h, : len(kept)] = p0[s, h, kept]
    assert torch.equal(k, wk) and torch.equal(v, wv)
    assert torch.equal(m1.view(torch.int32), wm.view(torch.int32)) and torch.equal(p1, wp)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lens,keep,sink,recent", [
    ([1], 1, 0, 0), ([2], 1, 0, 0), ([0, 1, 5], 3, 1, 1), ([448, 300, 100], 200, 4, 32), ([1500], 750, 0, 0),
    ([1500, 40], 1499, 1000, 499), ([700, 701], 1, 0, 1), ([65, 64, 63], 64, 0, 64), ([5000, 33], 1023, 1, 1)])
def test_evict_matches_rule(R, in_place, dtype, lens, keep, sink, recent):
    _evict_case(R, lens, 64, dtype, keep, sink, recent, in_place=in_place, seed=keep)


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("page", [1, 7, 16, 100, 1500])
@pytest.mark.parametrize("layout", ["head", "token"])
def test_evict_page_sizes_layouts_and_odd_masses(R, in_place, page, layout):
    _evict_case(R, [333, 200, 91], page, BF, 120, 3, 11, in_place=in_place, layout=layout, seed=page, odd=True)


def test_evict_to_fresh_pages_with_masses_in_place(R):
    """The rows go to other pages while the masses, labels and lengths are updated where they are."""
    torch.manual_seed(3)
    k = torch.randn(80, 2, 64, 64, device="cuda").to(BF)
    table = torch.arange(40, dtype=torch.int32, device="cuda").reshape(2, 20).contiguous()
    fresh = torch.arange(40, 80, dtype=torch.int32, device="cuda").reshape(2, 20).contiguous()
    k0, mass = k.clone(), torch.rand(2, 2, 1280, device="cuda")
    pos = torch.randint(0, 1 << 30, mass.shape, dtype=torch.int32, device="cuda")
    m0, p0 = mass.clone(), pos.clone()
    kv_len = torch.tensor([1280, 900], dtype=torch.int32, device="cuda")
    R.PagedCache(k, k.clone(), table).evict(kv_len, mass, keep=850, max_kv=1280, recent=3, page_table_out=fresh, pos=pos)
    torch.cuda.synchronize()
    assert kv_len.tolist() == [850, 850]
    for s in range(2):
        for h in range(2):
            kept = torch.tensor(evict_rule(m0[s, h].cpu(), (1280, 900)[s], 850, 0, 3), device="cuda")
            assert torch.equal(mass[s, h, :850], m0[s, h, kept]) and torch.equal(pos[s, h, :850], p0[s, h, kept])
            assert torch.equal(mass[s, h, 850:], m0[s, h, 850:])
            rows = k[fresh[s].long(), h].reshape(-1, 64)[:850]
            assert torch.equal(rows, k0[table[s].long(), h].reshape(-1, 64)[kept])


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("lens,hkv,page", [([9000], 1, 64), ([3000, 2999], 2, 16), ([30000, 12345, 500], 2, 100)])
def test_evict_shared_by_a_cluster(R, in_place, lens, hkv, page):
    """Few long caches: several CTAs select for one (request, head)."""
    _evict_case(R, lens, page, BF, max(lens) // 3, 2, 7, hkv=hkv, in_place=in_place, seed=page, odd=True)


@pytest.mark.parametrize("in_place", [False, True])
def test_evict_long(R, in_place):
    _evict_case(R, [70001], 64, BF, 20000, 4, 100, hkv=1, in_place=in_place, seed=5)


def test_evict_equal_masses_keep_the_first(R):
    lens, keep = [1000], 300
    k = torch.randn(16, 1, 64, 64, device="cuda")
    table = torch.arange(16, dtype=torch.int32, device="cuda")[None].contiguous()
    pos = torch.zeros(1, 1, keep, dtype=torch.int32, device="cuda")
    for value in (0.0, 1.0, math.nan, -3.0, math.inf):
        cache = R.PagedCache(k.clone(), k.clone(), table)
        kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")
        mass = torch.full((1, 1, 1000), value, device="cuda")
        cache.evict(kv_len, mass, keep=keep, max_kv=1000, recent=10, pos_out=pos)
        torch.cuda.synchronize()
        assert pos[0, 0].tolist() == list(range(290)) + list(range(990, 1000))


def test_evict_slots_bad_ids_and_bad_pages(R):
    k = torch.randn(20, 2, 16, 64, device="cuda").to(BF)
    v = torch.randn(20, 2, 16, 64, device="cuda").to(BF)
    table = torch.randperm(20)[:20].reshape(4, 5).to(torch.int32).cuda()
    table[2, 1] = 77                                          # positions 16..31 of slot 2 have no page
    k0 = k.clone()
    cache = R.PagedCache(k, v, table)
    kv_len = torch.tensor([80, 80, 80, 80], dtype=torch.int32, device="cuda")
    mass = torch.rand(4, 2, 80, device="cuda")
    m0 = mass.clone()
    req = torch.tensor([2, -1, 0, 9], dtype=torch.int32, device="cuda")
    cache.evict(kv_len, mass, keep=50, max_kv=80, req_ids=req)
    torch.cuda.synchronize()
    assert kv_len.tolist() == [50, 80, 50, 80]
    assert torch.equal(mass[[1, 3]], m0[[1, 3]])
    for s in (1, 3):
        assert torch.equal(k[table[s].long()], k0[table[s].long()])
    for h in range(2):
        kept = evict_rule(m0[2, h].cpu(), 80, 50, 0, 0)
        want = k0.clone()
        for j, src in enumerate(kept):
            if j // 16 != 1 and src // 16 != 1:
                want[table[2, j // 16], h, j % 16] = k0[table[2, src // 16], h, src % 16]
        rows = table[2, [0, 2, 3, 4]].long()
        assert torch.equal(k[rows, h], want[rows, h])


def test_evict_in_a_graph_and_twice(R):
    k = torch.randn(30, 2, 16, 64, device="cuda").to(BF)
    table = torch.arange(24, dtype=torch.int32, device="cuda").reshape(2, 12).contiguous()
    kv_len = torch.tensor([180, 60], dtype=torch.int32, device="cuda")
    mass = torch.rand(2, 2, 192, device="cuda")
    a, b = k.clone(), k.clone()
    ref = R.PagedCache(a, a.clone(), table)
    l1, m1 = kv_len.clone(), mass.clone()
    ref.evict(l1, m1, keep=100, max_kv=192, sink=2, recent=9)
    cache = R.PagedCache(b, b.clone(), table)
    l2, m2 = torch.zeros_like(kv_len), mass.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        cache.evict(l2, m2, keep=100, max_kv=192, sink=2, recent=9)
    l2.copy_(kv_len)
    for _ in range(3):                                        # the second and third replay find a cache that fits
        g.replay()
    torch.cuda.synchronize()
    assert l1.tolist() == l2.tolist() == [100, 60]
    assert torch.equal(a, b) and torch.equal(m1, m2)


# ------------------------------------------------------------------ logits rules
def _rules_case(n, H, V, hist=0, window=0, pen=True, bias=0, masks=0, seed=0, special=False):
    g = np.random.default_rng(seed)
    c = dict(z=(g.standard_normal((n, H, V)) * 3).astype(np.float32))
    hot = g.integers(0, V, max(1, V // 20))
    c["history"] = g.choice(hot, (n, hist)).astype(np.int32) if hist else None
    c["hist_len"] = g.integers(0, hist + 1, n).astype(np.int32) if hist else None
    c["block"] = g.choice(hot, (n, H + 2)).astype(np.int32)
    c["block_len"] = g.integers(0, H + 1, n).astype(np.int32)
    c["block_len"][0] = H
    c["window"] = window
    c["rep"], c["pres"], c["freq"] = ((1 + g.random(n) * 0.5).astype(np.float32), g.random(n).astype(np.float32),
                                      (g.random(n) - 0.3).astype(np.float32)) if pen else (None, None, None)
    c["bias"] = None
    if bias:
        ids = np.where(g.random((n, bias)) < 0.4, g.choice(hot, (n, bias)), g.integers(-2, V + 2, (n, bias))).astype(np.int32)
        c["bias"] = (ids, (g.standard_normal((n, bias)) * 4).astype(np.float32), g.integers(0, bias + 1, n).astype(np.int32))
        c["bias"][2][0] = bias
    c["masks"] = c["mask_row"] = None
    if masks:
        words = (V + 31) // 32
        m = g.integers(0, 1 << 32, (masks, words), dtype=np.uint64).astype(np.uint32)
        m[-1] = 0                                             # a state that allows nothing
        if masks > 1:
            m[0] = 0
            t = int(g.integers(0, V))
            m[0, t // 32] = np.uint32(1) << np.uint32(t % 32)  # and one that forces a token
        c["masks"], c["mask_row"] = m, g.integers(-2, masks + 2, (n, H)).astype(np.int32)
    if special:
        r = g.random(c["z"].shape)
        c["z"][r < 0.02] = -np.inf
        c["z"][(r > 0.02) & (r < 0.03)] = np.finfo(np.float32).min
        c["z"][(r > 0.03) & (r < 0.05)] = -0.0
        c["z"][0, 0, :: max(1, V // 7)] = np.inf
        if masks:
            c["z"][(r > 0.5) & (r < 0.51)] = np.nan
            dead = np.isnan(c["z"]).any((0, 1))               # NaN only where every state excludes it
            for w in range(c["masks"].shape[1]):
                for b in range(32):
                    if w * 32 + b < V and dead[w * 32 + b]:
                        c["masks"][:, w] &= ~np.uint32(1 << b)
            c["mask_row"] = np.clip(c["mask_row"], 0, masks - 1)
    return c


def _dev(x):
    return None if x is None else torch.as_tensor(np.ascontiguousarray(x.view(np.int32) if x.dtype == np.uint32 else x)).cuda()


def _rules_check(R, c, in_place=False, pad=0, shift=0):
    n, H, V = c["z"].shape
    b = c["bias"]
    rules = R.LogitsRules(_dev(c["rep"]), _dev(c["pres"]), _dev(c["freq"]), c["window"], *(map(_dev, b) if b else (None,) * 3),
                          masks=_dev(c["masks"]))
    store = torch.full((n * H * (V + pad) + 8,), 3.0, device="cuda")
    z = store[shift: shift + n * H * (V + pad)].view(n, H, V + pad)[:, :, :V]
    z.copy_(torch.as_tensor(c["z"]))
    out = z if in_place else torch.full((n, H, V), 9.0, device="cuda")
    target = torch.full((n, H), 77, dtype=torch.int32, device="cuda")
    lp = torch.full((n, H), 77.0, device="cuda")
    rules.apply(z, _dev(c["history"]), _dev(c["hist_len"]), _dev(c["block"]), _dev(c["block_len"]), _dev(c["mask_row"]),
                out=out, target=target, logprob=lp)
    torch.cuda.synchronize()
    w_out, w_t, w_lp = rules_rule(c["z"], c["history"], c["hist_len"], c["block"], c["block_len"], c["window"], c["rep"],
                                  c["pres"], c["freq"], b, c["masks"], c["mask_row"])
    got = out.cpu().numpy()
    for i in range(n):
        m = int(c["block_len"][i])
        np.testing.assert_array_equal(got[i, :m], w_out[i, :m])
        rest = c["z"][i, m:] if in_place else np.full_like(got[i, m:], 9.0)
        np.testing.assert_array_equal(got[i, m:], rest)
        assert target[i].tolist() == [int(x) for x in w_t[i]]
        # each pass sums 32 values per thread, five steps across the warp, and three merges of up to eight parts;
        # an exponential is good to 2^-20, the logarithm to two steps
        passes = max(1, -(-V // 65536))
        tol = (passes * 40 + 16) * 2.0 ** -24 + 2.0 ** -19
        g, w = lp[i].double().cpu().numpy(), w_lp[i]
        assert np.array_equal(np.isinf(g), np.isinf(w))
        f = np.isfinite(w)
        assert np.all(np.abs(g[f] - w[f]) <= tol * (1 + np.abs(w[f]))), (g, w)
    if pad:                                                   # between the rows nothing is written
        assert bool((store[shift: shift + n * H * (V + pad)].view(n, H, V + pad)[:, :, V:] == 3.0).all())


@pytest.mark.parametrize("V", [1, 2, 31, 33, 1000, 8192, 8193, 51865, 51866, 65536, 70001])
def test_rules_vocabularies(R, V):
    _rules_check(R, _rules_case(3, 4, V, hist=20, bias=6, masks=3, seed=V))


@pytest.mark.parametrize("kw", [dict(), dict(hist=50), dict(hist=50, window=1), dict(hist=50, window=7), dict(hist=9, window=100),
                                dict(pen=False, bias=5), dict(pen=False, masks=3), dict(pen=False), dict(hist=300, bias=40, masks=5),
                                dict(hist=2000, window=1500)])
@pytest.mark.parametrize("n,H", [(1, 1), (5, 9)])
def test_rules_parts(R, kw, n, H):
    _rules_check(R, _rules_case(n, H, 1000, seed=3, **kw))


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("pad,shift", [(0, 0), (0, 1), (3, 2), (5, 3), (4, 0)])
@pytest.mark.parametrize("V", [997, 20001])
def test_rules_strides_and_alignment(R, in_place, pad, shift, V):
    _rules_check(R, _rules_case(2, 3, V, hist=30, bias=3, masks=2, seed=pad), in_place=in_place, pad=pad, shift=shift)


@pytest.mark.parametrize("V", [500, 30000])
@pytest.mark.parametrize("masks", [0, 4])
def test_rules_infinities_and_masked_nans(R, V, masks):
    _rules_check(R, _rules_case(3, 5, V, hist=30, bias=4, masks=masks, seed=V + masks, special=True))


def test_rules_bad_token_ids_ignored(R):
    c = _rules_case(2, 3, 500, hist=12, bias=4, masks=2, seed=1)
    c["history"][:, ::3] = -1
    c["history"][:, 1::3] = 500
    c["block"][:, 1] = 1 << 30
    c["hist_len"][:] = (-4, 99)
    _rules_check(R, c)


def test_rules_many_rows(R):
    _rules_check(R, _rules_case(40, 9, 3001, hist=64, bias=8, masks=4, seed=5))


def test_rules_nan_is_never_chosen(R):
    z = torch.tensor([[[math.nan, 1.0, math.nan, 4.0]]], device="cuda")
    t, lp = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.zeros(1, 1, device="cuda")
    R.LogitsRules().apply(z, target=t, logprob=lp)
    torch.cuda.synchronize()
    assert t.item() == 3 and math.isnan(lp.item())


def test_rules_captured_reads_the_state_at_replay(R):
    V = 2000
    z0 = torch.randn(2, 3, V, device="cuda")
    hist = torch.zeros(2, 10, dtype=torch.int32, device="cuda")
    hl = torch.zeros(2, dtype=torch.int32, device="cuda")
    rules = R.LogitsRules(repetition=torch.full((2,), 2.0, device="cuda"))
    out, t = torch.zeros_like(z0), torch.zeros(2, 3, dtype=torch.int32, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rules.apply(z0, hist, hl, out=out, target=t)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, z0)
    hist[:, 0] = z0[:, 0].argmax(1).int()
    hl.fill_(1)
    g.replay()
    torch.cuda.synchronize()
    for i in range(2):
        v = int(hist[i, 0])
        x = z0[i, 0, v]
        assert out[i, 0, v] == (x / 2 if x > 0 else x * 2) and t[i, 0] == out[i, 0].argmax()


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("dtype", [BF, F32])
def test_attend_evict_attend(R, dtype):
    """Chunks accumulate weights, the cache is cut to its heaviest positions, and the next tokens attend to what is
    left: the same as attention over the kept positions picked by hand."""
    c = AttnCase([60, 30], [260, 190], hq=4, hkv=2, dtype=dtype, page=16, seed=21)
    cache = R.PagedCache(c.k, c.v, c.table)
    mass = torch.zeros_like(c.mass0)
    cache.attend(c.q, c.kv_len, c.cu, max_q=60, max_kv=c.max_kv, mass=mass, out=torch.empty_like(c.q))
    kept = [[evict_rule(mass[s, h].cpu(), c.slot_len[s], 100, 2, 20) for h in range(2)] for s in range(2)]
    old = [[(c.k[c.table[s].long()].transpose(1, 2).reshape(-1, 2, 64)[kept[s][h], h].double(),
             c.v[c.table[s].long()].transpose(1, 2).reshape(-1, 2, 64)[kept[s][h], h].double()) for h in range(2)] for s in range(2)]
    cache.evict(c.kv_len, mass, keep=100, max_kv=c.max_kv, sink=2, recent=20)
    q = (torch.randn(2, 4, 64, device="cuda") * 1.5).to(dtype)
    cu = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    out = cache.attend(q, c.kv_len, cu, max_q=1, max_kv=100)
    torch.cuda.synchronize()
    assert c.kv_len.tolist() == [100, 100]
    for s in range(2):
        for u in range(4):
            k, v = old[s][u // 2]
            w = torch.softmax(k @ q[s, u].double() * 0.125, 0)
            want = w @ v
            rel = 2.0 ** -7 if dtype is BF else 2.0 ** -16    # the weights' and the output's rounding; fp32 sums
            assert bool(((out[s, u].double() - want).abs() <= rel * (w @ v.abs())).all())

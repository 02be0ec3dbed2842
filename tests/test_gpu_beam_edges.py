"""The beam-search serving operators on the GPU where their number formats end:
scale bytes at both ends of their range, values whose product with the scale
passes fp32, and what rows that do not see such blocks must not feel."""
import math
import subprocess
import sys

import numpy as np
import pytest
import torch

from beam_common import D, Pool, Q8Case
from test_gpu_beam_operators import DT, R, check_q8, i32, run_append  # noqa: F401  (R: the fixture)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ append
@pytest.mark.parametrize("byte", [0, 1, 100, 246, 247, 252, 253, 254])
@pytest.mark.parametrize("block", [8, 96])
def test_append_to_blocks_of_any_scale(R, byte, block):
    """Blocks begun before the call, of the smallest scale to the largest: rows from nothing up to 2^127."""
    def values(x):
        x = x.clone()
        for r in range(len(x)):
            x[r] *= 2.0 ** [0, -140, -126, -60, 60, 110, 120, 124, 125, 126][r % 10]
        return x.clamp(-2.0 ** 127, 2.0 ** 127)
    for first in range(1, 8):
        pool = Pool(1, 3, 2, block, DT["e4m3"], block, seed=first)
        pool.scales[:] = byte
        run_append(R, pool, [block + 5], [first + block + 5], 2, "none", with_q=False, values=values, seed=first)
        pool.scales[:] = byte
        run_append(R, pool, [2], [first + 2], 2, "none", with_q=False, values=values, seed=first)


# ------------------------------------------------------------------ what a row does not see
@pytest.mark.parametrize("c,hq", [(2, 1), (9, 1), (16, 2), (5, 6)])
@pytest.mark.parametrize("block,L", [(8, 265), (8, 281), (16, 273), (32, 257), (64, 1665)])
@pytest.mark.parametrize("gap", [24, 60, 140, 200])
def test_attend_8bit_scale_that_a_row_does_not_see(R, c, hq, block, L, gap):
    """A block that starts with the last position, which the chunk's last row alone sees, and whose values' scale is
    2^gap of the others': the other rows' bits are those without it."""
    cs = Q8Case([c], [L], hq, 1, 64, block=block, spread=0, seed=c + L)
    cs.scales[1] -= 70                                     # values of 2^-70, scales of about 2^-78
    cs.v.mul_(2.0 ** -70)
    cache = cs.cache(R)

    def attend():
        lse = torch.zeros(cs.q.shape[:2], device="cuda")
        out = cache.attend(cs.q, cs.kv_len, cs.cu, max_q=c, max_kv=L, lse=lse)
        torch.cuda.synchronize()
        return out[: cs.rows].clone(), lse[: cs.rows].clone()
    want = attend()
    cs.scales[1][cs.table[0, (L - 1) // 64], :, (L - 1) % 64 // block] += gap
    got = attend()
    for a, b in zip(got, want):
        assert torch.equal(a[: c - 1], b[: c - 1])
    assert torch.equal(got[1], want[1])
    assert gap == 200 or bool(torch.isfinite(got[0]).all())           # values of 2^122 may pass fp32 in the sums
    assert bool((got[0][c - 1] != want[0][c - 1]).any())


def test_attend_8bit_scales_that_grow_along_a_chunk(R):
    """The last blocks' scales are far larger, one after the other: each row is as exact as what it sees allows."""
    c, L, block = 24, 288, 8
    cs = Q8Case([c], [L], 2, 1, 16, block=block, spread=0, seed=4)
    up = torch.zeros(L // block, dtype=torch.int64)
    up[-3:] = torch.tensor([30, 60, 90])                   # rows of the chunk see none, one, two or all of them
    for e in range(L // 16):
        for b in range(2):
            f = int(up[2 * e + b])
            page = int(cs.table[0, e])
            cs.scales[1, page, :, b] += np.uint8(f % 256)
            cs.v[page, :, b * block: (b + 1) * block] *= 2.0 ** f
    (o, l, _), (to, tl, _) = cs.reference()
    out = cs.cache(R).attend(cs.q, cs.kv_len, cs.cu, max_q=c, max_kv=L)
    torch.cuda.synchronize()
    got = out[: cs.rows].double().cpu()
    v = cs.v.double().cpu()[cs.table[0].long().cpu()].transpose(1, 2).reshape(-1, D)
    for t in range(c):
        # the weights' last step, as for whole caches (check_q8), of what this row sees
        lim = L - c + t + 1
        floor = 2.0 ** -30 * lim * 2 * float(v[:lim].abs().max())
        assert bool(((got[t] - o[t]).abs() <= to[t] + floor).all()), t


@pytest.mark.parametrize("n,hkv,c", [(1, 1, 60), (1, 2, 100), (2, 1, 300), (60, 3, 60)])
@pytest.mark.parametrize("page,block", [(64, 16), (64, 8), (48, 48)])
@pytest.mark.parametrize("code,scale", [(0x78, 247), (0xFE, 247), (0x7E, 254), (0xF1, 248)])
def test_attend_8bit_infinite_values_stay_where_they_are_seen(R, n, hkv, c, page, block, code, scale):
    """Elements whose value passes fp32 (256 * 2^120, as an append of finite rows may leave it) in a position that the
    last row alone sees, in one head of one request: that row's element is infinite, and nothing else differs."""
    L = 6 * 96 + 1                                         # a block of its own in every page size
    cs = Q8Case([c] * n, [L] * n, hkv, hkv, page, block=block, seed=c)
    at = int(cs.table[n - 1, (L - 1) // page]), hkv - 1, (L - 1) % page
    codes = cs.v8.view(torch.uint8)
    codes[at] = 0
    cache = cs.cache(R)

    def attend():
        return cache.attend(cs.q, cs.kv_len, cs.cu, max_q=c, max_kv=L)[: cs.rows].clone()
    want = attend()
    codes[at[0], at[1], at[2], 7] = code
    cs.scales[1][at[0], at[1], at[2] // block] = scale
    got = attend()
    torch.cuda.synchronize()
    hit = torch.zeros_like(got, dtype=torch.bool)
    hit[n * c - 1, hkv - 1, 7] = True
    assert torch.equal(got[~hit], want[~hit])
    assert float(got[hit]) == (-math.inf if code & 0x80 else math.inf)


def test_attend_8bit_infinite_values_of_both_signs(R):
    """Rows that see none, one or both of them."""
    c, L = 100, 401
    cs = Q8Case([c], [L], 1, 1, 16, block=16, seed=1)
    codes = cs.v8.view(torch.uint8)
    cache = cs.cache(R)
    for pos in (384, 400):
        codes[int(cs.table[0, pos // 16]), 0, :] = 0
    want = cache.attend(cs.q, cs.kv_len, cs.cu, max_q=c, max_kv=L)[:c].clone()
    for pos, code in ((384, 0x7C), (400, 0xFC)):
        page = int(cs.table[0, pos // 16])
        codes[page, 0, 0, 3] = code
        cs.scales[1][page] = 250
    got = cache.attend(cs.q, cs.kv_len, cs.cu, max_q=c, max_kv=L)[:c]
    torch.cuda.synchronize()
    others = [d for d in range(D) if d != 3]
    assert torch.equal(got[:, 0, others], want[:, 0, others])
    assert torch.equal(got[:83], want[:83])                # row r sees 302 + r positions
    assert bool((got[83:99, 0, 3] == math.inf).all()) and bool(torch.isnan(got[99, 0, 3]))


# ------------------------------------------------------------------ the description of a cache
# One that is not in 8 bits, as long as it was before there were caches in 8 bits, at the very end of a mapping: what
# the library reads behind it ends the process on the host.
SHORT = """
import ctypes as C, mmap, sys
sys.path.insert(0, {root!r})
import torch
from speculative_whisper_asr_gb300 import binding as B, runtime as R
libc = C.CDLL(None)
libc.mmap.restype = C.c_void_p
libc.mmap.argtypes = [C.c_void_p, C.c_size_t, C.c_int, C.c_int, C.c_int, C.c_long]
libc.mprotect.argtypes = [C.c_void_p, C.c_size_t, C.c_int]
size, page = B.PagedCacheDesc.k_scale.offset, mmap.PAGESIZE
at = libc.mmap(None, 2 * page, mmap.PROT_READ | mmap.PROT_WRITE, mmap.MAP_PRIVATE | mmap.MAP_ANONYMOUS, -1, 0)
assert at not in (None, C.c_void_p(-1).value) and libc.mprotect(at + page, page, 0) == 0
class Short:
    def __init__(self, desc):
        C.memmove(at + page - size, C.addressof(desc), size)
C_addressof = C.addressof
B.C.addressof = lambda x: at + page - size if isinstance(x, Short) else C_addressof(x)
def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")
torch.manual_seed(0)
state = []
for short in (False, True):
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn(6, 2, 16, 64, generator=g).to(torch.{dtype}).cuda() for _ in range(2))
    rows = torch.randn(3, 8, 64, generator=g).to(torch.{dtype}).cuda()
    cache = R.PagedCache(k, v, i32(0, 1, 2, 3, 4, 5).view(2, 3))
    if short:
        cache.desc = Short(cache.desc)
    L, cu = i32(20, 20), i32(0, 2, 3)
    mass = torch.rand(2, 2, 48, generator=g).cuda()
    cache.append(rows[:, :2], rows[:, 2:4], L, cu, max_q=2)
    out = cache.attend(rows[:, 4:].contiguous(), L, cu, max_q=2, max_kv=20, mass=mass)
    if short:
        a = cache._reorder
        a.n_req, a.beams, a.req_ids, a.kv_len, a.page_table = 1, 2, 0, L.data_ptr(), 0
        parent = i32(1, 1)
        a.parent = parent.data_ptr()
        B.ws_cache_reorder(cache.desc, a, torch.cuda.current_stream().cuda_stream)
    else:
        cache.reorder(i32(1, 1).view(1, 2), L, table=False)
    cache.evict(L, mass, keep=10, max_kv=20)
    torch.cuda.synchronize()
    state.append([k, v, rows, out, mass, L])
assert all(torch.equal(a, b) for a, b in zip(*state))
print("done")
"""


@pytest.mark.parametrize("dtype", ["bfloat16", "float32"])
def test_scales_of_other_caches_are_not_read(R, dtype):
    import __graft_entry__ as g
    r = subprocess.run([sys.executable, "-c", SHORT.format(root=g.ROOT, dtype=dtype)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "done" in r.stdout, (r.returncode, r.stderr[-1500:])


# ------------------------------------------------------------------ two heads per CTA, in parts
@pytest.mark.parametrize("n,hkv,page,block,causal", [(31, 5, 64, 16, True), (31, 5, 16, 8, False), (77, 2, 64, 64, True),
                                                     (52, 3, 48, 16, False), (52, 3, 64, 8, True)])
def test_attend_8bit_single_row_tiles_of_many_in_parts(R, n, hkv, page, block, causal):
    """More heads in all than SMs (odd numbers of them too) over caches long enough to be split: short, empty and full
    requests beside each other."""
    kv = 1550
    chunks = [[64, 49, 3, 0, 1, 57][i % 6] if i < 12 else 1 + i % 2 for i in range(n)]
    lens = [max(c, [kv, 1200, 0 if not c else 5, 700, kv - 1, 130][i % 6]) for i, c in enumerate(chunks)]
    check_q8(R, Q8Case(chunks, lens, hkv, hkv, page, block=block, causal=causal, seed=n + hkv))


@pytest.mark.parametrize("heads", [[0], [1], [4]])
@pytest.mark.parametrize("block", [16, 8])
def test_attend_8bit_values_that_are_not_finite_in_parts(R, heads, block):
    """NaN and infinite values in the first and the last part, in some heads of a pair: those rows of those heads."""
    n, hkv, c, L = 31, 5, 60, 1553
    cs = Q8Case([c] * n, [L] * n, hkv, hkv, 16, block=block, seed=5)
    codes = cs.v8.view(torch.uint8)
    first, late = L - c + 9, L - 1                         # seen from row 9 on, and by the last row
    for pos in (first, late):
        codes[int(cs.table[n - 2, pos // 16]), :, pos % 16] = 0
    cache = cs.cache(R)

    def attend():
        return cache.attend(cs.q, cs.kv_len, cs.cu, max_q=c, max_kv=L)[: cs.rows].clone()
    want = attend()
    for h in heads:
        codes[int(cs.table[n - 2, first // 16]), h, first % 16, 7] = 0x7F
        page = int(cs.table[n - 2, late // 16])
        codes[page, h, late % 16, 9] = 0xFE
        cs.scales[1][page, h, late % 16 // block] = 250
    got = attend()
    torch.cuda.synchronize()
    row0 = (n - 2) * c
    nan, inf = (torch.zeros_like(got, dtype=torch.bool) for _ in range(2))
    nan[row0 + 9: row0 + c, heads, 7] = True
    inf[row0 + c - 1, heads, 9] = True
    # what else the last block holds has another scale now, which rows that see it feel
    felt = torch.zeros_like(nan)
    felt[row0 + c - 1 - (late % 16 % block): row0 + c, heads] = True
    assert bool(torch.isnan(got)[nan].all()) and bool((got[inf] == -math.inf).all())
    assert torch.equal(got[~nan & ~inf & ~felt], want[~nan & ~inf & ~felt])

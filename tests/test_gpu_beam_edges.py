"""The beam-search serving operators on the GPU where their number formats end:
scale bytes at both ends of their range, values whose product with the scale
passes fp32, and what rows that do not see such blocks must not feel."""
import math

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
@pytest.mark.parametrize("gap", [24, 60, 140])
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
    assert bool(torch.isfinite(got[0]).all()) and torch.equal(got[1], want[1])
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

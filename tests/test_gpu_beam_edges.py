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

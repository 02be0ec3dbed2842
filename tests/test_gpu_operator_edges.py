"""Where the decode-serving operators meet odd inputs: rows that hold nothing
next to rows that do, NaN beside sound values, calls of several heights,
refused calls between sound ones, grammars that depend on the tokens or leave
none."""
import math

import numpy as np
import pytest
import torch

import synth
from gpu_common import dev_i32, small_shape
from operator_common import E32, AttnCase, close, evict_rule

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def R():
    import __graft_entry__ as g
    g.build()
    from speculative_whisper_asr_gb300 import runtime
    return runtime


def _attend(R, c, mass=True, lse=True, cache=None):
    cache = cache or R.PagedCache(c.k, c.v, c.table)
    out = torch.full_like(c.q, 7.0)
    ls = torch.full(c.q.shape[:2], 7.0, device="cuda") if lse else None
    ms = c.mass0.clone() if mass else None
    cache.attend(c.q, c.kv_len, c.cu, max_q=c.max_q, max_kv=c.max_kv, causal=c.causal, scale=c.scale, out=out, lse=ls,
                 mass=ms, req_ids=c.req)
    torch.cuda.synchronize()
    return out, ls, ms


def _decoder(R, dtype, n=2, frames=(140, 90), max_frames=None, drafter=True, **kw):
    s = small_shape(dtype, **kw)
    tw = synth.target_weights(s, 3)
    dw = synth.drafter_weights(s, 3, tw) if drafter else None
    dec = R.Decoder(s, tw, dw, max_batch=max(n, 2), max_frames=max_frames or max(frames))
    req = dec.slots(list(range(n)))
    A = [synth.encoder_states(s, 3, i, frames=f) for i, f in enumerate(frames[:n])]
    dec.cross_kv(req, torch.cat([dec.enc_tensor(a) for a in A]), list(frames[:n]))
    return s, dec, req, A


# ------------------------------------------------------------------ rows that hold nothing
@pytest.mark.parametrize("G,c", [(3, 40), (5, 70), (6, 300), (7, 9), (40, 11), (2, 70)])
@pytest.mark.parametrize("causal", [True, False])
def test_rows_that_hold_nothing_do_not_change_the_others(R, G, c, causal):
    """Long chunks whose row tiles are not full: the same call gives the same bits whatever ran before it and
    whatever stands in the rows of q behind the chunk."""
    x = AttnCase([c], [900], hq=2 * G, hkv=2, causal=causal, seed=G, spare_rows=130)
    dirt = AttnCase([256], [300], hq=1, hkv=1, causal=False, seed=1)
    clean = AttnCase([256], [300], hq=1, hkv=1, causal=False, seed=1)
    dirt.q.fill_(math.nan)
    clean.q.zero_()
    runs = []
    for before, tail in ((clean, 0.0), (dirt, 0.0), (clean, math.nan), (clean, 1e30), (dirt, -1e30)):
        x.q_all[x.rows:] = tail
        for _ in range(20):                                   # on every SM
            _attend(R, before, mass=False)
        runs.append([t[: x.rows] if k < 2 else t for k, t in enumerate(_attend(R, x))])
    for other in runs[1:]:
        for a, b in zip(runs[0], other):
            assert torch.equal(a, b)


def test_a_request_does_not_change_with_the_next_one(R):
    """A partial row tile reaches into the next request's rows of q."""
    x = AttnCase([70, 60], [900, 700], hq=6, hkv=2, causal=False, seed=4)
    a = _attend(R, x)
    x.q[70:130] = math.nan
    b = _attend(R, x)
    for k in (0, 1):
        assert torch.equal(a[k][:70], b[k][:70])
    assert torch.equal(a[2][0], b[2][0])

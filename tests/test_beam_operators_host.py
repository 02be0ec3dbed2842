"""Refusals of the beam-search serving operators: every bad argument is
reported on the host before anything is enqueued (no GPU needed)."""
import math

import numpy as np
import pytest

from beam_common import e4m3_round, e4m3_value, needed_exponent


@pytest.fixture(scope="module")
def B():
    import __graft_entry__ as g
    g.build()
    from speculative_whisper_asr_gb300 import binding
    return binding


def _cache(B, **kw):
    a = dict(dtype=B.WS_E4M3, n_kv_heads=4, page_size=64, n_pages=10, k=4096, v=8192, page_stride=4 * 64 * 64,
             head_stride=64 * 64, token_stride=64, page_table=4096, n_slots=15, table_stride=7, k_scale=4096, v_scale=8192,
             scale_page_stride=16, scale_head_stride=4, scale_block=16)
    a.update(kw)
    return B.PagedCacheDesc(**a)


def _append(B, **kw):
    a = dict(n_req=2, req_ids=0, kv_len=4096, cu_q=4096, total_q=8, max_q=4, k=1 << 20, k_stride=256, v=2 << 20, v_stride=256,
             n_heads=8, q=3 << 20, q_stride=512, q_out=4 << 20, q_out_stride=512, turns=4096, rot_dims=64, rot_halves=0, pos=0)
    a.update(kw)
    return B.AppendArgs(**a)


def _reorder(B, **kw):
    a = dict(n_req=3, beams=5, req_ids=0, kv_len=4096, parent=4096, page_table=4096)
    a.update(kw)
    return B.ReorderArgs(**a)


def _beam(B, **kw):
    a = dict(n=3, beams=5, vocab=1000, logits=4096, ld=1000, eos_id=7, score=1 << 20, score_out=2 << 20, parent=4096, token=8192,
             tokens=3 << 20, tokens_out=4 << 20, length=5 << 20, length_out=6 << 20, capacity=448, max_done=5, n_done=7 << 20,
             n_done_out=8 << 20, done_score=9 << 20, done_length=10 << 20, done_tokens=11 << 20)
    a.update(kw)
    return B.BeamArgs(**a)


def _attn(B, **kw):
    a = dict(n_req=2, req_ids=0, kv_len=4096, cu_q=4096, total_q=8, max_q=4, max_kv=448, n_heads=8, causal=1,
             scale=0.125, q=4096, q_stride=512, out=1 << 20, out_stride=512, lse=0, mass=0, mass_stride=0)
    a.update(kw)
    return B.AttentionArgs(**a)


def _refused(B, fn, code):
    with pytest.raises(B.WSError) as e:
        fn()
    assert e.value.code == code, e.value
    assert B.ws_last_error()


@pytest.mark.parametrize("bad", [dict(dtype=3), dict(k_scale=0), dict(v_scale=0), dict(scale_block=0), dict(scale_block=-4),
                                 dict(scale_block=24), dict(scale_block=128), dict(scale_page_stride=3), dict(scale_head_stride=3),
                                 dict(scale_head_stride=-4), dict(scale_page_stride=1 << 31), dict(scale_head_stride=1 << 31),
                                 dict(token_stride=72), dict(page_stride=4 * 64 * 64 + 8), dict(head_stride=8), dict(k=4104)])
def test_bad_8bit_cache_refused(B, bad):
    c = _cache(B, **bad)
    assert B.ws_paged_attention_workspace(c, _attn(B)) == 0
    _refused(B, lambda: B.ws_paged_attention(c, _attn(B), 4096, 1 << 40, 0), B.WS_EINVAL)
    _refused(B, lambda: B.ws_cache_append(c, _append(B), 0), B.WS_EINVAL)
    _refused(B, lambda: B.ws_cache_reorder(c, _reorder(B), 0), B.WS_EINVAL)


def test_what_8bit_caches_do_not_have(B):
    """No accumulated weights, no eviction."""
    a = _attn(B, mass=4096, mass_stride=448)
    assert B.ws_paged_attention_workspace(_cache(B), a) == 0
    _refused(B, lambda: B.ws_paged_attention(_cache(B), a, 4096, 1 << 40, 0), B.WS_EUNSUPPORTED)
    e = B.EvictArgs(n_req=2, kv_len=4096, kv_len_out=4096, max_kv=448, keep=200, mass=4096, mass_stride=448)
    assert B.ws_cache_evict_workspace(_cache(B), e) == 0
    _refused(B, lambda: B.ws_cache_evict(_cache(B), e, 4096, 1 << 40, 0), B.WS_EUNSUPPORTED)


@pytest.mark.parametrize("bad", [dict(n_req=-1), dict(n_req=65536), dict(total_q=-1), dict(max_q=-1), dict(max_q=(1 << 28) + 1),
                                 dict(kv_len=0), dict(cu_q=0), dict(k=0), dict(v=0), dict(q_out=0), dict(q=0), dict(n_heads=0),
                                 dict(n_heads=65536, q_stride=1 << 23, q_out_stride=1 << 23), dict(k=(1 << 20) + 8), dict(v=(2 << 20) + 2),
                                 dict(q=(3 << 20) + 4), dict(q_out=(4 << 20) + 8), dict(k_stride=248), dict(v_stride=252),
                                 dict(q_stride=511), dict(q_out_stride=504), dict(k_stride=1 << 37), dict(rot_dims=0),
                                 dict(rot_dims=12), dict(rot_dims=72), dict(rot_halves=2), dict(turns=4100), dict(n_req=16),
                                 # the turned queries over other queries, keys or values
                                 dict(q_out=3 << 20, q_out_stride=1024), dict(q_out=(3 << 20) + 16), dict(q_out=1 << 20),
                                 dict(q_out=(2 << 20) - 16), dict(q_out=(1 << 20) + 512, q_out_stride=1024, k_stride=512),
                                 dict(k=(3 << 20) + 1024, k_stride=768, q=3 << 20, q_stride=768, q_out=(3 << 20) + 16, q_out_stride=768)])
def test_bad_append_refused(B, bad):
    _refused(B, lambda: B.ws_cache_append(_cache(B), _append(B, **bad), 0), B.WS_EINVAL)


@pytest.mark.parametrize("bad", [dict(n_req=-1), dict(n_req=65536), dict(beams=0), dict(beams=17), dict(kv_len=0), dict(parent=0),
                                 dict(page_table=8192), dict(n_req=4)])
def test_bad_reorder_refused(B, bad):
    _refused(B, lambda: B.ws_cache_reorder(_cache(B), _reorder(B, **bad), 0), B.WS_EINVAL)


@pytest.mark.parametrize("bad", [dict(n=-1), dict(beams=0), dict(beams=17), dict(vocab=0, ld=1), dict(vocab=(1 << 18) + 1, ld=1 << 20),
                                 dict(n=20000), dict(eos_id=-2), dict(eos_id=1000), dict(max_done=-1), dict(logits=0),
                                 dict(logits=4098), dict(ld=999), dict(score=0), dict(score_out=0), dict(parent=0), dict(token=0),
                                 dict(tokens_out=0), dict(length=0), dict(length_out=0), dict(capacity=0), dict(tokens=0),
                                 dict(n_done_out=0), dict(done_score=0), dict(n_done=0),
                                 dict(score_out=(1 << 20) + 4), dict(tokens_out=(3 << 20) + 448 * 4), dict(length_out=(5 << 20) - 4),
                                 dict(n_done_out=(7 << 20) + 8), dict(done_tokens=3 << 20), dict(done_tokens=(4 << 20) + 4)])
def test_bad_beam_refused(B, bad):
    a = _beam(B, **bad)
    assert B.ws_beam_select_workspace(a) == 0
    _refused(B, lambda: B.ws_beam_select(a, 4096, 1 << 40, 0), B.WS_EINVAL)


def test_beam_workspace_checked(B):
    a = _beam(B)
    need = B.ws_beam_select_workspace(a)
    assert need >= 15 * 6 * 8
    _refused(B, lambda: B.ws_beam_select(a, 4096, need - 1, 0), B.WS_ENOSPACE)
    _refused(B, lambda: B.ws_beam_select(a, 0, need, 0), B.WS_EINVAL)
    _refused(B, lambda: B.ws_beam_select(a, 4104, need, 0), B.WS_EINVAL)
    # every size has one: candidates of all parts of all rows
    for n, beams, vocab in ((1, 1, 1), (1, 16, 1 << 18), (4095, 16, 51866), (96, 5, 51866)):
        assert B.ws_beam_select_workspace(_beam(B, n=n, beams=beams, vocab=vocab, ld=vocab, eos_id=-1, tokens=0, tokens_out=0, length=0,
                                                length_out=0, n_done=0, n_done_out=0, done_score=0, done_length=0,
                                                done_tokens=0)) >= n * beams * (beams + 2) * 8


def test_null_structs_refused(B):
    assert B.lib.ws_cache_append(None, None, None) == B.WS_EINVAL
    assert B.lib.ws_cache_reorder(None, None, None) == B.WS_EINVAL
    assert B.lib.ws_beam_select(None, None, 0, None) == B.WS_EINVAL
    assert B.lib.ws_beam_select_workspace(None) == 0


def test_empty_calls_do_nothing(B):
    B.ws_cache_append(_cache(B), _append(B, n_req=0), 0)
    B.ws_cache_append(_cache(B), _append(B, total_q=0), 0)
    B.ws_cache_append(_cache(B), _append(B, max_q=0), 0)
    B.ws_cache_reorder(_cache(B), _reorder(B, n_req=0), 0)
    B.ws_cache_reorder(_cache(B), _reorder(B, beams=1), 0)
    B.ws_beam_select(_beam(B, n=0), 0, 0, 0)


def test_the_rules_of_the_gpu_tests():
    """e4m3 as its 16 exponents and 8 significands define it; the scale of a block at its border."""
    c = np.arange(256)
    v = e4m3_value(c)
    assert v[0x7E] == 448.0 and v[0x08] == 2.0 ** -6 and v[0x01] == 2.0 ** -9 and v[0x38] == 1.0 and v[0xB8] == -1.0
    assert np.isnan(v[0x7F]) and np.isnan(v[0xFF])
    fin = v[np.isfinite(v)]
    assert np.array_equal(e4m3_round(fin), fin)
    mids = (np.unique(fin)[1:] + np.unique(fin)[:-1]) / 2
    assert np.all(np.isin(e4m3_round(mids), fin))
    assert math.isnan(e4m3_round(np.inf)) and e4m3_round(1.0625) == 1.0 and e4m3_round(1.1875) == 1.25
    assert needed_exponent(448.0) == 0 and needed_exponent(448.0 * (1 + 2 ** -20)) == 1 and needed_exponent(0.0) == -127

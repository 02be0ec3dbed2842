"""Refusals of the operators on a caller's own buffers: every bad argument is
reported on the host before anything is enqueued (no GPU needed)."""
import pytest


@pytest.fixture(scope="module")
def B():
    import __graft_entry__ as g
    g.build()
    from speculative_whisper_asr_gb300 import binding
    return binding


def _cache(B, **kw):
    a = dict(dtype=B.WS_BF16, n_kv_heads=4, page_size=64, n_pages=10, k=4096, v=8192, page_stride=4 * 64 * 64,
             head_stride=64 * 64, token_stride=64, page_table=4096, n_slots=3, table_stride=7)
    a.update(kw)
    return B.PagedCacheDesc(**a)


def _attn(B, **kw):
    a = dict(n_req=2, req_ids=0, kv_len=4096, cu_q=4096, total_q=8, max_q=4, max_kv=448, n_heads=8, causal=1,
             scale=0.125, q=4096, q_stride=512, out=8192, out_stride=512, lse=0, mass=0, mass_stride=0)
    a.update(kw)
    return B.AttentionArgs(**a)


def _evict(B, **kw):
    a = dict(n_req=2, req_ids=0, kv_len=4096, kv_len_out=4096, max_kv=448, keep=200, sink=2, recent=10, mass=4096,
             mass_stride=448, mass_out=0, mass_out_stride=0, pos=0, pos_stride=0, pos_out=0, pos_out_stride=0,
             page_table_out=0, table_out_stride=0)
    a.update(kw)
    return B.EvictArgs(**a)


def _rules(B, **kw):
    a = dict(n=2, H=3, vocab=1000, logits=4096, ld=1000, out=8192, ld_out=1000, block_len=0, history=0, hist_len=0,
             hist_stride=0, block=0, block_stride=0, window=0, repetition=0, presence=0, frequency=0, bias_ids=0,
             bias_vals=0, bias_len=0, bias_stride=0, masks=0, n_masks=0, mask_row=0, target=4096, logprob=4096)
    a.update(kw)
    return B.RulesArgs(**a)


def _refused(B, fn, code):
    with pytest.raises(B.WSError) as e:
        fn()
    assert e.value.code == code, e.value
    assert B.ws_last_error()


BAD_CACHE = [dict(dtype=2), dict(n_kv_heads=0), dict(n_kv_heads=65536), dict(page_size=0), dict(n_pages=0), dict(k=0),
             dict(v=0), dict(k=4104), dict(v=4098), dict(page_stride=-8), dict(page_stride=100), dict(head_stride=4),
             dict(head_stride=0), dict(page_stride=0), dict(token_stride=68), dict(token_stride=56), dict(token_stride=0), dict(page_table=0), dict(n_slots=0),
             dict(table_stride=0), dict(page_stride=1 << 37)]


@pytest.mark.parametrize("bad", BAD_CACHE)
def test_bad_cache_refused(B, bad):
    c = _cache(B, **bad)
    assert B.ws_paged_attention_workspace(c, _attn(B)) == 0
    assert B.ws_cache_evict_workspace(c, _evict(B)) == 0
    _refused(B, lambda: B.ws_paged_attention(c, _attn(B), 4096, 1 << 40, 0), B.WS_EINVAL)
    _refused(B, lambda: B.ws_cache_evict(c, _evict(B), 4096, 1 << 40, 0), B.WS_EINVAL)


@pytest.mark.parametrize("bad", [dict(n_req=-1), dict(n_req=65536), dict(total_q=-1), dict(max_q=-1), dict(max_kv=-1),
                                 dict(n_heads=0), dict(n_heads=6), dict(causal=2), dict(scale=float("nan")),
                                 dict(scale=float("inf")), dict(kv_len=0), dict(cu_q=0), dict(q=0), dict(out=0),
                                 dict(q=4104), dict(out=8200), dict(q_stride=504), dict(out_stride=516),
                                 dict(mass=4096, mass_stride=447), dict(n_req=4)])
def test_bad_attention_refused(B, bad):
    a = _attn(B, **bad)
    assert B.ws_paged_attention_workspace(_cache(B), a) == 0
    _refused(B, lambda: B.ws_paged_attention(_cache(B), a, 4096, 1 << 40, 0), B.WS_EINVAL)


@pytest.mark.parametrize("bad", [dict(n_req=-1), dict(max_kv=0), dict(keep=0), dict(keep=449), dict(sink=-1),
                                 dict(recent=-1), dict(sink=150, recent=51), dict(kv_len=0), dict(kv_len_out=0),
                                 dict(mass=0), dict(mass_stride=447), dict(mass_out=8192, mass_out_stride=199),
                                 dict(mass_out=4096, mass_out_stride=449), dict(pos=4096, pos_stride=447),
                                 dict(pos_out=4096, pos_out_stride=199),
                                 dict(pos=4096, pos_stride=448, pos_out=4096, pos_out_stride=449),
                                 dict(page_table_out=8192, table_out_stride=0),
                                 dict(page_table_out=8192, table_out_stride=3), dict(n_req=4)])
def test_bad_eviction_refused(B, bad):
    a = _evict(B, **bad)
    assert B.ws_cache_evict_workspace(_cache(B), a) == 0
    _refused(B, lambda: B.ws_cache_evict(_cache(B), a, 4096, 1 << 40, 0), B.WS_EINVAL)


def test_workspaces_checked(B):
    need = B.ws_cache_evict_workspace(_cache(B), _evict(B))
    assert need >= 2 * 4 * 200 * 4
    _refused(B, lambda: B.ws_cache_evict(_cache(B), _evict(B), 4096, need - 1, 0), B.WS_ENOSPACE)
    _refused(B, lambda: B.ws_cache_evict(_cache(B), _evict(B), 0, need, 0), B.WS_EINVAL)
    _refused(B, lambda: B.ws_cache_evict(_cache(B), _evict(B), 4097, need, 0), B.WS_EINVAL)
    a = _attn(B, mass=4096, mass_stride=448)
    need = B.ws_paged_attention_workspace(_cache(B), a)
    assert need > 0
    _refused(B, lambda: B.ws_paged_attention(_cache(B), a, 4096, need - 1, 0), B.WS_ENOSPACE)
    _refused(B, lambda: B.ws_paged_attention(_cache(B), a, 0, need, 0), B.WS_EINVAL)


@pytest.mark.parametrize("bad", [dict(n=-1), dict(H=-1), dict(H=16385), dict(vocab=0), dict(vocab=(1 << 18) + 1, ld=1 << 25, ld_out=1 << 25),
                                 dict(logits=0), dict(out=0), dict(logits=4097), dict(out=4098), dict(ld=999),
                                 dict(ld_out=999), dict(out=4096, ld_out=1001), dict(history=4096, hist_stride=8),
                                 dict(hist_stride=-1), dict(block=4096, block_stride=2),
                                 dict(window=-1), dict(bias_ids=4096, bias_stride=4),
                                 dict(bias_ids=4096, bias_vals=4096, bias_stride=4), dict(bias_stride=-1),
                                 dict(masks=4096, n_masks=0, mask_row=4096), dict(masks=4096, n_masks=2),
                                 dict(n=1 << 30, H=4)])
def test_bad_rules_refused(B, bad):
    _refused(B, lambda: B.ws_logits_rules(_rules(B, **bad), 0), B.WS_EINVAL)


def test_rules_too_many_listed_tokens_refused(B):
    _refused(B, lambda: B.ws_logits_rules(_rules(B, history=4096, hist_len=4096, hist_stride=4097), 0), B.WS_EUNSUPPORTED)
    _refused(B, lambda: B.ws_logits_rules(_rules(B, history=4096, hist_len=4096, hist_stride=4000, window=3000, bias_ids=4096,
                                                 bias_vals=4096, bias_len=4096, bias_stride=1097), 0), B.WS_EUNSUPPORTED)


def test_null_structs_refused(B):
    assert B.lib.ws_paged_attention(None, None, None, 0, None) == B.WS_EINVAL
    assert B.lib.ws_cache_evict(None, None, None, 0, None) == B.WS_EINVAL
    assert B.lib.ws_logits_rules(None, None) == B.WS_EINVAL
    assert B.lib.ws_paged_attention_workspace(None, None) == 0
    assert B.lib.ws_cache_evict_workspace(None, None) == 0


def test_empty_calls_do_nothing(B):
    B.ws_paged_attention(_cache(B), _attn(B, n_req=0), 0, 0, 0)
    B.ws_paged_attention(_cache(B), _attn(B, total_q=0), 0, 0, 0)
    B.ws_cache_evict(_cache(B), _evict(B, n_req=0), 0, 0, 0)
    B.ws_logits_rules(_rules(B, n=0), 0)
    B.ws_logits_rules(_rules(B, H=0), 0)


@pytest.mark.parametrize("q,qs,out,os_", [
    (4096, 512, 4096, 512),                              # in place
    (4096, 512, 4096 + 512, 512),                        # half a row behind
    (4096 + 1024 * 7, 512, 4096, 512),                   # out ends in q's first row
    (4096, 1024, 4096 + 1024 + 16, 1024),                # interleaved rows of one buffer that reach into the next
    (4096, 1024, 4096 + 1024 - 16, 1024),
    (4096 + 2048 * 3 + 16, 1024, 4096 + 1024, 1024),
    (4096 + 4096, 1024, 4096, 512),                      # other strides, ranges that meet
])
@pytest.mark.parametrize("dtype", [0, 1])
def test_out_over_q_refused(B, q, qs, out, os_, dtype):
    """8 rows of 8 heads (1,024 bytes in bf16; strides in elements) that share elements with q."""
    f = 2 if dtype == B.WS_F32 else 1                    # fp32: the same picture with every distance doubled
    a = _attn(B, q=q * f, q_stride=qs, out=out * f, out_stride=os_)
    _refused(B, lambda: B.ws_paged_attention(_cache(B, dtype=dtype), a, 4096, 1 << 40, 0), B.WS_EINVAL)


@pytest.mark.parametrize("ld,out,ld_out", [(1000, 4096 + 4, 1000), (1000, 4096 + 4000, 1000), (1000, 4096 + 4000 * 6 - 4, 1000),
                                           (2000, 4096 + 4000 - 4, 2000), (2000, 4096 + 4000 + 4, 2000), (2000, 4096 + 4000, 1000)])
def test_rules_out_partly_over_logits_refused(B, ld, out, ld_out):
    """6 rows of 1,000 logits (4,000 bytes)."""
    _refused(B, lambda: B.ws_logits_rules(_rules(B, ld=ld, out=out, ld_out=ld_out), 0), B.WS_EINVAL)

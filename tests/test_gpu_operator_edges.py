"""Where the decode-serving operators meet odd inputs: rows that hold nothing
next to rows that do, NaN beside sound values, calls of several heights,
refused calls between sound ones, grammars that depend on the tokens or leave
none."""
import math

import numpy as np
import pytest
import torch

import synth
from gpu_common import dev_i32, small_shape, teacher_forced_logits
from operator_common import E32, AttnCase, close

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


# ------------------------------------------------------------------ a grammar that leaves no token
def _allow_all_or_nothing(R, s):
    words = (s.vocab + 31) // 32
    m = np.zeros((2, words), np.uint32)
    m[0] = 0xFFFFFFFF                                         # state 0: every token, state 1: none
    return R.LogitsRules(masks=torch.as_tensor(m.view(np.int32)).cuda())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("mode,where", [(m, w) for m in ("ar", "spec", "sample-ar", "sample-spec") for w in ("prompt", "first")]
                         + [("spec", "later"), ("sample-spec", "later")])    # rows behind the first: speculative rounds alone
def test_a_state_without_tokens_ends_the_request(R, dtype, mode, where):
    """Request 0 reaches a grammar state that excludes every token: it ends there, with what it had, and the status
    word says so.  Request 1 goes on as if alone."""
    n, budget = 2, 12
    s, dec, req, _ = _decoder(R, dtype, n)
    sampling, spec = mode.startswith("sample"), mode.endswith("spec")

    def run(dead):
        b = dec.new_batch(req, [budget] * n, sampling=sampling, rules=_allow_all_or_nothing(R, s))
        P = len(s.prompt)
        for H in (1, P, s.K + 1):
            b.states(H).fill_(0)
        if dead and where == "prompt":
            b.states(P)[0] = 1
        elif dead and where == "first":
            b.states(1)[0] = 1
            b.states(s.K + 1)[0] = 1
        elif dead:
            b.states(s.K + 1)[0, 2:] = 1                      # the third row and those after it
        if spec:
            rounds = R.run_spec(dec, b, temperature=0.9 if sampling else 0.0, seed=3, max_rounds=200)
        elif sampling:
            rounds = R.run_ar_sampling(dec, b, 0.9, 3, max_rounds=200)
        else:
            rounds = R.run_ar(dec, b, max_rounds=200)
        assert rounds < 200
        return b

    full = run(False)
    assert dec.status() == 0
    want = full.transcripts()
    b = run(True)
    got = b.transcripts()
    assert got[1] == want[1]
    assert all(0 <= t < s.vocab for t in got[0])
    assert got[0] == want[0][: len(got[0])]
    if where == "prompt":
        assert got[0] == []
    elif where == "first":
        assert len(got[0]) == 1
    assert b.done.tolist() == [1, 1] and b.blen.tolist() == [0, 0]
    ended_early = len(got[0]) < len(want[0])
    assert ended_early or where == "later"
    assert dec.status() == (16 if ended_early else 0)
    assert b.budget[0].item() == budget - len(got[0])
    # the slots decode on afterwards
    again = run(False)
    assert again.transcripts() == want and dec.status() == 0


# ------------------------------------------------------------------ a grammar that depends on the tokens
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("sampling", [False, True])
def test_grammar_states_follow_the_proposals(R, dtype, sampling):
    """The state of a row is given by the token before it: speculative decoding obeys the grammar at every token, and
    greedy decoding gives the autoregressive transcript."""
    n, budget = 2, 40
    s, dec, req, _ = _decoder(R, dtype, n)
    g = np.random.default_rng(5)
    words = (s.vocab + 31) // 32
    m = g.integers(0, 1 << 32, (4, words), dtype=np.uint64).astype(np.uint32)     # half of the tokens after each
    rules = R.LogitsRules(masks=torch.as_tensor(m.view(np.int32)).cuda())
    seen = []

    def next_states(batch, block, block_len, states):
        seen.append(tuple(states.shape))
        if block is None:                                     # the prompt: the transcript is empty
            states.fill_(3)
        else:                                                 # column j is the token before row j
            assert block.shape == states.shape and block_len.shape == (n,)
            states.copy_(block % 3)

    def run(spec, **kw):
        b = dec.new_batch(req, [budget] * n, sampling=sampling, rules=rules, next_states=next_states)
        if spec:
            R.run_spec(dec, b, temperature=0.8 if sampling else 0.0, seed=2, **kw)
        elif sampling:
            R.run_ar_sampling(dec, b, 0.8, 2)
        else:
            R.run_ar(dec, b)
        tr = b.transcripts()
        for t in tr:
            assert len(t) == budget or t[-1] == s.eos_id
            for j, tok in enumerate(t):
                state = 3 if j == 0 else t[j - 1] % 3
                assert (int(m[state, tok // 32]) >> (tok % 32)) & 1, (j, tok)
        return tr

    ar = run(False)
    assert (n, len(s.prompt)) in seen and (n, 1) in seen
    for kw in (dict(), dict(k_verify=3), dict(graph=False)):
        sp = run(True, **kw)
        if not sampling:
            assert sp == ar
    assert (n, s.K + 1) in seen and (n, 4) in seen
    assert dec.status() == 0


def test_next_states_needs_masks(R):
    s, dec, req, _ = _decoder(R, "f32", 1)
    with pytest.raises(ValueError):
        dec.new_batch(req, [4], next_states=lambda *a: None)
    with pytest.raises(ValueError):
        dec.new_batch(req, [4], rules=R.LogitsRules(), next_states=lambda *a: None)


# ------------------------------------------------------------------ refused calls between sound ones
def test_rules_after_a_refused_batch_size(R):
    """A batch of another size is refused; the next sound call still has its biases, penalties and masks."""
    V = 500
    z = torch.randn(2, 1, V, device="cuda")
    ids = torch.tensor([[3], [4]], dtype=torch.int32, device="cuda")
    vals = torch.full((2, 1), 50.0, device="cuda")
    lens = torch.ones(2, dtype=torch.int32, device="cuda")
    masks = torch.full((1, (V + 31) // 32), -1, dtype=torch.int32, device="cuda")
    masks[0, 0] = ~(1 << 7)
    row = torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    for kw in (dict(bias_ids=ids, bias_vals=vals, bias_len=lens), dict(bias_ids=ids, bias_vals=vals, bias_len=lens, masks=masks)):
        rules = R.LogitsRules(**kw)
        state = row if "masks" in kw else None
        a = rules.apply(z, mask_row=state, out=torch.empty_like(z))
        with pytest.raises(ValueError):
            rules.apply(torch.randn(3, 1, V, device="cuda"))
        with pytest.raises(ValueError):                       # another vocabulary: the masks do not fit
            rules.apply(torch.randn(3, 1, 2 * V, device="cuda"))
        b = rules.apply(z, mask_row=state, out=torch.empty_like(z))
        torch.cuda.synchronize()
        assert a[0, 0, 3] == z[0, 0, 3] + 50.0 and torch.equal(a, b)


# ------------------------------------------------------------------ accumulated frame weights in the decoder
def _rows(dec, s, req, block, one_by_one):
    """Target logits of the block's rows: in one verify, or row by row with a forced accept after each."""
    import speculative_whisper_asr_gb300.binding as B
    stream = torch.cuda.current_stream().cuda_stream
    n, H = block.shape
    dec.reset(req)
    b = dec.new_batch(req, [10 ** 6] * n)
    out = []
    for part in ([block[:, j: j + 1].contiguous() for j in range(H)] if one_by_one else [block]):
        h = part.shape[1]
        t, lg = torch.zeros(n, h, dtype=torch.int32, device="cuda"), torch.zeros(n, h, s.vocab, device="cuda")
        bl = dev_i32([h] * n)
        dec.verify(req, part, bl, t, lg)
        a = b._args(B.WS_ACCEPT_FORCED, h, part, bl, t, b.block1, b.blen)
        B.ws_accept(dec.ctx, n, req.data_ptr(), a, stream)
        out.append(lg)
    torch.cuda.synchronize()
    return torch.cat(out, 1)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("frames", [(140, 90, 33), (1500, 700, 1), (2600, 300, 40)])
def test_rows_do_not_depend_on_the_call(R, dtype, accumulate, frames):
    """A row's logits are the same bits in a block and alone, with other requests and without, also while the frames'
    weights are accumulated."""
    s, dec, req, _ = _decoder(R, dtype, 3, frames, drafter=False)
    block = torch.as_tensor(np.random.default_rng(7).integers(0, s.vocab, (3, 9)), dtype=torch.int32, device="cuda")
    dec.accumulate_frames(accumulate)
    whole = _rows(dec, s, req, block, False)
    assert torch.equal(_rows(dec, s, req, block, True), whole)
    for i in range(3):
        one = dec.slots([i])
        assert torch.equal(_rows(dec, s, one, block[i: i + 1], False)[0], whole[i])
    for H in (2, 8):
        assert torch.equal(_rows(dec, s, req, block[:, :H].contiguous(), False), whole[:, :H])


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_speculative_equals_autoregressive_while_accumulating(R, dtype):
    s, dec, req, _ = _decoder(R, dtype, 2, (1400, 900), max_pos=448)
    dec.accumulate_frames(True)
    a, b = dec.new_batch(req, [150, 150]), dec.new_batch(req, [150, 150])
    R.run_ar(dec, a)
    R.run_spec(dec, b)
    assert a.transcripts() == b.transcripts()


# ------------------------------------------------------------------ NaN beside sound values
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("c,lens", [(1, (300, 130)), (6, (300, 130)), (16, (70, 33)), (30, (300, 130)), (90, (300, 130)),
                                    (9, (2500, 64)), (5, (5000, 64))])
def test_a_nan_row_adds_its_weights_only_where_it_sees(R, dtype, c, lens):
    """The NaN of one query row reaches the masses of the positions that row sees, of its KV head and request, and no
    other position."""
    x = AttnCase([c, c], lens, dtype=dtype, hq=4, hkv=2, page=16, seed=c)
    t = c // 2
    sound = AttnCase([c, c], lens, dtype=dtype, hq=4, hkv=2, page=16, seed=c)
    x.table[0, 1] = -1                                        # positions 16..31 of the first cache have no page
    sound.table[0, 1] = -1
    tol = sound.reference(bad_pages=(1,))[1][2]               # of request 0 alone: the other has its second page
    clean = _attend(R, sound)[2]
    x.q[t, 2, 5] = math.nan                                   # row t of request 0, KV head 1
    mass = _attend(R, x)[2]
    L = lens[0]
    sees = torch.zeros(mass.shape, dtype=torch.bool, device="cuda")
    sees[0, 1, : L - c + t + 1] = True
    sees[0, 1, 16:32] = False
    assert bool(mass[sees].isnan().all())
    assert not bool(mass[~sees].isnan().any())
    assert torch.equal(mass[0, :, 16:32], x.mass0[0, :, 16:32])
    other = torch.ones_like(sees)
    other[0, 1] = False
    assert torch.equal(mass[other], clean[other])             # other heads and requests: untouched
    behind = ~sees
    behind &= ~other
    close("positions that the row does not see", mass[behind], clean[behind].double().cpu(), 2 * tol[behind.cpu()])


# ------------------------------------------------------------------ log probabilities of large logits
@pytest.mark.parametrize("size", [30.0, 100.0, 1e3, 1e4, 1e6, -1e3, -1e4])
@pytest.mark.parametrize("n,V", [(2, 1000), (3, 51866), (200, 5001)])
def test_log_probabilities_far_from_zero(R, size, n, V):
    """Every logit shifted: the log probability of the largest does not lose what the shift's size rounds away."""
    g = np.random.default_rng(int(abs(size)) + V)
    z = (g.standard_normal((n, 1, V)) + size).astype(np.float32)
    forced = g.integers(0, V, n)
    bias = np.where(np.arange(n) % 2 == 0, 3.0, abs(size)).astype(np.float32)      # odd rows: a certain token
    rules = R.LogitsRules(bias_ids=dev_i32(forced[:, None]), bias_vals=torch.as_tensor(bias[:, None]).cuda(),
                          bias_len=dev_i32(np.ones(n)))
    lp, out = torch.zeros(n, 1, device="cuda"), torch.empty(n, 1, V, device="cuda")
    rules.apply(torch.as_tensor(z).cuda(), out=out, target=torch.zeros(n, 1, dtype=torch.int32, device="cuda"), logprob=lp)
    torch.cuda.synchronize()
    y = out[:, 0].double().cpu()
    want = y.max(1).values - torch.logsumexp(y, 1)
    got = lp[:, 0].double().cpu()
    assert bool((got <= 0).all())
    # differences of logits are exact to half a step, their product with log2(e) to two, an exponential to 2^-20; a
    # thread's sum has at most V / 512 terms and the joins 16 more
    d = (y.max(1).values[:, None] - y).clamp(max=100.0)
    w = torch.softmax(y, 1)
    tol = (w * d).sum(1) * 4 * E32 + 2.0 ** -20 + (V // 512 + 32) * E32 + want.abs() * 4 * E32
    assert bool(((got - want).abs() <= tol).all()), float(((got - want).abs() / tol).max())


# ------------------------------------------------------------------ calls with nothing to see
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("chunks,lens", [([1], [4000]), ([1, 1], [9000, 9000]), ([9, 9], [3000, 3000]), ([50, 20], [700, 513])])
def test_empty_caches_then_the_next_kernel(R, dtype, chunks, lens):
    """Every cache empty: the rows are zero for whatever is enqueued next, in a captured graph too, and no mass moves."""
    x = AttnCase(chunks, lens, dtype=dtype, hq=4, hkv=2, seed=3)
    x.kv_len.zero_()
    cache = R.PagedCache(x.k, x.v, x.table)
    out, seen, mass = torch.empty_like(x.q), torch.empty_like(x.q), x.mass0.clone()
    lse = torch.empty(x.q.shape[:2], device="cuda")

    def calls():
        out.fill_(7.0)
        cache.attend(x.q, x.kv_len, x.cu, max_q=x.max_q, max_kv=x.max_kv, out=out, lse=lse, mass=mass)
        seen.copy_(out)
        out.fill_(9.0)

    calls()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls()
    for _ in range(50):
        g.replay()
    torch.cuda.synchronize()
    assert bool((seen[: x.rows] == 0).all()) and bool((seen[x.rows:] == 7.0).all()) and bool((out == 9.0).all())
    assert bool((lse[: x.rows] == -math.inf).all()) and torch.equal(mass, x.mass0)


# ------------------------------------------------------------------ outputs beside and over inputs
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("c", [3, 30, 100])
def test_out_beside_q_in_the_same_rows(R, dtype, c):
    """q and out as columns of one buffer; out over q is refused."""
    x = AttnCase([c], [140], hq=4, hkv=4, dtype=dtype, seed=9)
    wide = torch.zeros(c, 12, 64, device="cuda", dtype=dtype)
    wide[:, 4:8] = x.q[:c]
    want, tol = x.reference()
    cache = R.PagedCache(x.k, x.v, x.table)
    args = dict(kv_len=x.kv_len, cu_q=x.cu, max_q=c, max_kv=140)
    cache.attend(wide[:, 4:8], out=wide[:, 8:12], **args)
    torch.cuda.synchronize()
    close("out", wide[:, 8:12], want[0], tol[0])
    assert torch.equal(wide[:, 4:8], x.q[:c])
    for out in (wide[:, 4:8], wide[:, 5:9], wide[:, 2:6]):
        with pytest.raises(R.B.WSError) as e:
            cache.attend(wide[:, 4:8], out=out, **args)
        assert e.value.code == R.B.WS_EINVAL
    both = torch.zeros(2 * c + 2, 4, 64, device="cuda", dtype=dtype)       # q directly before and behind out
    for at in (0, c):
        both[at: at + c] = x.q[:c]
        cache.attend(both[at: at + c], out=both[c - at: 2 * c - at], **args)
        torch.cuda.synchronize()
        close("out", both[c - at: 2 * c - at], want[0], tol[0])
    with pytest.raises(R.B.WSError):
        cache.attend(both[:c], out=both[c - 1: 2 * c - 1], **args)


def test_rules_out_beside_logits(R):
    """New logits in the other half of the rows' buffer."""
    both = torch.randn(2, 3, 2000, device="cuda")
    z, out = both[:, :, :1000], both[:, :, 1000:]
    want = z.clone()
    R.LogitsRules().apply(z, out=out)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(z, want)
    with pytest.raises(R.B.WSError):
        R.LogitsRules().apply(z, out=both[:, :, 999:1999])


# ------------------------------------------------------------------ a context's scratch
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K,frames,n", [(1, 4096, 2), (1, 2100, 3), (12, 4096, 2), (15, 1, 2), (1, 64, 70)])
def test_the_smallest_and_largest_contexts_hold_their_scratch(R, dtype, K, frames, n):
    """Frame weights and the largest cut in contexts whose blocks are short and caches long, and the other way round."""
    s = small_shape(dtype, n_layers=1, K=K, prompt=(990,) * min(2, K + 1), hist_layers=(0,))
    dec = R.Decoder(s, synth.target_weights(s, 3), None, max_batch=n, max_frames=frames, max_block=K + 1)
    req = dec.slots(list(range(n)))
    A = synth.encoder_states(s, 3, 0, frames=frames)
    dec.cross_kv(req, torch.cat([dec.enc_tensor(A)] * n), [frames] * n)
    block = torch.full((n, K + 1), 5, dtype=torch.int32, device="cuda")
    t, bl = torch.zeros_like(block), dev_i32([K + 1] * n)
    lg = torch.zeros(n, K + 1, s.vocab, device="cuda")
    dec.accumulate_frames(True)
    dec.verify(req, block, bl, t, lg)
    torch.cuda.synchronize()
    total = dec.frame_mass().double().sum(-1)
    assert bool((total - (K + 1)).abs().max() < (K + 1) * (2.0 ** -19 + 4096 * 2.0 ** -24))
    assert torch.equal(lg, lg[:1].expand_as(lg))              # the same request n times
    if frames > 1:
        dec.evict_frames(req, frames - 1)
    again = torch.zeros_like(lg)
    dec.reset(req)
    dec.verify(req, block, bl, t, again)
    torch.cuda.synchronize()
    assert torch.equal(again, again[:1].expand_as(lg)) and bool(torch.isfinite(again).all())
    assert dec.status() == 0


# ------------------------------------------------------------------ what a cache object holds
def test_a_growing_loop_holds_nothing_per_step(R):
    """A decoding loop whose length grows by one: the object keeps no entry per step, and its scratch fits every call."""
    x = AttnCase([1], [400], hq=4, hkv=2, seed=3)
    cache = R.PagedCache(x.k, x.v, x.table)
    mass = torch.zeros_like(x.mass0)

    def held():
        return sum(len(v) for v in vars(cache).values() if isinstance(v, (dict, list)))

    sizes = []
    for L in range(1, 400):
        x.kv_len.fill_(L)
        out = cache.attend(x.q[:1], x.kv_len, x.cu, max_q=1, max_kv=L, mass=mass)
        sizes.append(held())
    torch.cuda.synchronize()
    assert sizes[-1] <= sizes[20] + 6                         # scratch that was outgrown, at doubling sizes
    want, tol = x.reference()
    x.kv_len.fill_(400)
    out = cache.attend(x.q[:1], x.kv_len, x.cu, max_q=1, max_kv=400)
    close("out", out, want[0], tol[0])


# ------------------------------------------------------------------ readout after a cut
def test_readout_returns_with_the_full_caches(R):
    """While a slot's acoustic cache is cut there is no readout; once every cut slot has new acoustic keys there is."""
    s, dec, req, A = _decoder(R, "bf16", 2, (140, 90))
    dec.frame_mass().uniform_()
    dec.evict_frames(req, 50)

    def refused():
        with pytest.raises(R.B.WSError) as e:
            dec.set_readout(1, 10)
        return e.value.code == R.B.WS_EUNSUPPORTED

    assert refused()
    dec.cross_kv(dec.slots([1]), dec.enc_tensor(A[1]), [90])
    assert refused()                                          # slot 0 is still cut
    dec.cross_kv(dec.slots([0]), dec.enc_tensor(A[0]), [140])
    dec.set_readout(1, 10)
    b = dec.new_batch(req, [20, 20])
    R.run_spec(dec, b)
    dec.set_readout(-1, 0)
    plain = dec.new_batch(req, [20, 20])
    R.run_ar(dec, plain)
    assert b.transcripts() == plain.transcripts()
    dec.frame_mass().uniform_()
    dec.evict_frames(req, 139)                                # cuts slot 0 alone
    assert refused()


# ------------------------------------------------------------------ one-request contexts
def test_frames_in_a_one_request_context(R):
    """A bf16 context of one slot verifies in its dataflow kernel: weights are accumulated all the same, and over cut
    caches it gives what the kernel-per-operation path gives."""
    s = small_shape("bf16")
    tw = synth.target_weights(s, 3)
    dw = synth.drafter_weights(s, 3, tw)
    A = synth.encoder_states(s, 3, 0, frames=200)
    decs = [R.Decoder(s, tw, dw, max_batch=mb, max_frames=200) for mb in (1, 2)]
    got = []
    for dec in decs:
        req = dec.slots([0])
        dec.cross_kv(req, dec.enc_tensor(A), [200])
        tr = []
        for keep in (None, 60):
            b, c = dec.new_batch(req, [40]), dec.new_batch(req, [40])
            R.run_spec(dec, b, keep_frames=keep, evict_after=2)
            R.run_ar(dec, c)                                  # over the caches as they now are
            tr += [b.transcripts(), c.transcripts()]
            if keep is None:
                assert tr[0] == tr[1]
        d = dec.new_batch(req, [40])
        R.run_spec(dec, d)
        assert d.transcripts() == tr[3]
        assert dec.status() == 0
        got.append(tr)
    assert got[0][0] == got[1][0]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("spec", [False, True])
def test_keeping_every_frame_changes_nothing_beyond_the_tolerance(R, dtype, spec):
    """keep_frames as large as the caches: nothing is cut; a token differs from plain decoding only where the rounds
    that accumulated weights met logits closer than the model's tolerance."""
    s, dec, req, _ = _decoder(R, dtype, 2, (140, 90))
    run = R.run_spec if spec else R.run_ar
    plain, kept = dec.new_batch(req, [30, 30]), dec.new_batch(req, [30, 30])
    run(dec, plain)
    run(dec, kept, keep_frames=140, evict_after=3)
    rel = 1e-4 if dtype == "f32" else 2e-2
    for i, (a, b) in enumerate(zip(plain.transcripts(), kept.transcripts())):
        j = next((k for k in range(min(len(a), len(b))) if a[k] != b[k]), None)
        if j is None:
            assert a == b
            continue
        row = teacher_forced_logits(dec, dec.slots([i]), s, a[:j])[len(s.prompt) - 1 + j]
        assert row.max() - row[b[j]] <= 2 * rel * max(1.0, np.abs(row).max())
    again = dec.new_batch(req, [30, 30])
    run(dec, again)
    assert again.transcripts() == plain.transcripts()         # the caches are what they were


# ------------------------------------------------------------------ values that are not finite, where a row does not see
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("chunks,lens,hq,hkv,page", [
    ((5, 3), (300, 130), 4, 2, 64), ((16, 9), (70, 40), 2, 2, 16), ((30, 33), (300, 64), 2, 2, 64), ((40, 40), (200, 1025), 4, 4, 100),
    ((90, 70), (300, 130), 4, 2, 16), ((300, 128), (700, 500), 3, 3, 64), ((70, 1), (230, 90), 10, 2, 100),
    ((3, 2), (400, 300), 130, 1, 64), ((2, 3), (900, 300), 100, 1, 16), ((700,), (1500,), 5, 1, 128), ((60,), (5000,), 2, 1, 64),
    ((9,), (4000,), 1, 1, 64), ((100, 37), (100, 37), 2, 1, 7)])
def test_what_a_row_does_not_see_does_not_reach_it(R, dtype, chunks, lens, hq, hkv, page):
    """Values and keys of the chunk's own later positions that are not finite: rows before them are as with finite
    ones; rows that see an infinite or NaN value have it in that element alone."""
    x = AttnCase(chunks, lens, hq=hq, hkv=hkv, page=page, dtype=dtype, seed=sum(lens))
    clean = AttnCase(chunks, lens, hq=hq, hkv=hkv, page=page, dtype=dtype, seed=sum(lens))
    g = np.random.default_rng(sum(lens))
    inf = math.inf
    special = []                                              # (request, position, KV head, element, value)
    for i, (c, L) in enumerate(zip(chunks, lens)):
        first = max(0, L - c) + 1                             # the first position that some row does not see
        for pos in sorted(set(g.integers(first, L, 4).tolist() + [L - 1])) if first < L else []:
            h = int(g.integers(0, hkv))
            for e, v in zip(g.choice(64, 3, replace=False).tolist(), (inf, -inf, math.nan)):
                special.append((i, pos, h, e, v))
    for i, pos, h, e, v in special:
        p = int(x.table[i, pos // page])
        x.v[p, h, pos % page, e] = v
        clean.v[p, h, pos % page, e] = 0.0
    want, tol = clean.reference()
    out, lse, mass = _attend(R, x)
    ref = want[0].clone()
    row0 = np.concatenate([[0], np.cumsum(chunks)])
    G = hq // hkv
    for i, pos, h, e, v in special:
        first = pos - (lens[i] - chunks[i])                   # the first row of the chunk that sees pos
        rows = slice(row0[i] + max(0, first), row0[i + 1])
        ref[rows, h * G: (h + 1) * G, e] += v
    got = out[: x.rows].double().cpu()
    assert torch.equal(got.isnan(), ref.isnan())
    close("out", torch.nan_to_num(got, nan=0.0, posinf=inf, neginf=-inf), torch.nan_to_num(ref, nan=0.0, posinf=inf, neginf=-inf), tol[0])
    close("lse", lse[: x.rows], want[1], tol[1])
    close("mass", mass, want[2], tol[2])
    # a key
    y = AttnCase(chunks, lens, hq=hq, hkv=hkv, page=page, dtype=dtype, seed=sum(lens))
    want, tol = y.reference()
    i = len(chunks) - 1 if chunks[-1] > 1 else 0
    pos = lens[i] - 1 - (chunks[i] - 1) // 2
    y.k[int(y.table[i, pos // page]), 0, pos % page, 3] = math.nan
    out, lse, _ = _attend(R, y, mass=False)
    sees = slice(row0[i] + pos - (lens[i] - chunks[i]), row0[i + 1])
    assert bool(out[sees, :G].isnan().all()) and bool(lse[sees, :G].isnan().all())
    for a, w, t in ((out, want[0], tol[0]), (lse, want[1], tol[1])):
        a = a[: y.rows].double().cpu()
        a[sees, :G] = w[sees, :G]
        close("rows that do not see the key", a, w, t)

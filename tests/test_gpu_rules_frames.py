"""Logits rules and acoustic-cache eviction inside the decoding loop: the
speculative rounds reproduce the autoregressive ones under the same rules,
sampled tokens obey the grammar, verification's accumulated frame weights add
up, and a cut cache equals one that held only the kept frames."""
import numpy as np
import pytest
import torch

import synth
from gpu_common import dev_i32, logits_close, small_shape
from operator_common import rules_rule

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def R():
    import __graft_entry__ as g
    g.build()
    from speculative_whisper_asr_gb300 import runtime
    return runtime


def _decoder(R, dtype, n=2, frames=(140, 90), **kw):
    s = small_shape(dtype, **kw)
    tw = synth.target_weights(s, 3)
    dw = synth.drafter_weights(s, 3, tw)
    dec = R.Decoder(s, tw, dw, max_batch=max(n, 2), max_frames=max(frames))
    req = dec.slots(list(range(n)))
    A = [synth.encoder_states(s, 3, i, frames=f) for i, f in enumerate(frames[:n])]
    dec.cross_kv(req, torch.cat([dec.enc_tensor(a) for a in A]), list(frames[:n]))
    return s, dec, req, A


def _rules(R, s, n, masks=True, window=0):
    g = np.random.default_rng(11)
    rep = (1.1 + g.random(n) * 0.5).astype(np.float32)
    pres, freq = g.random(n).astype(np.float32), (0.5 * g.random(n)).astype(np.float32)
    ids = g.integers(0, s.vocab, (n, 12)).astype(np.int32)
    vals = (2.0 * g.standard_normal((n, 12))).astype(np.float32)
    lens = np.full(n, 12, np.int32)
    words = (s.vocab + 31) // 32
    m = (g.integers(0, 1 << 32, (n, words), dtype=np.uint64) | g.integers(0, 1 << 32, (n, words), dtype=np.uint64)).astype(np.uint32)
    host = dict(window=window, rep=rep, pres=pres, freq=freq, bias=(ids, vals, lens), masks=m if masks else None)
    c = lambda x: torch.as_tensor(x.view(np.int32) if x.dtype == np.uint32 else x).cuda()   # noqa: E731
    return host, R.LogitsRules(c(rep), c(pres), c(freq), window, c(ids), c(vals), c(lens), c(m) if masks else None)


def _set_states(b, s, n):
    for H in (1, len(s.prompt), s.K + 1):
        b.states(H).copy_(torch.arange(n, device="cuda", dtype=torch.int32)[:, None].expand(n, H))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("masks,window", [(False, 0), (True, 5)])
def test_rules_in_the_loop(R, dtype, masks, window):
    """Autoregressive decoding under rules equals the rules applied by hand to each step's logits, and speculative
    decoding equals autoregressive decoding."""
    n, budget = 2, 24
    s, dec, req, _ = _decoder(R, dtype, n)
    host, rules = _rules(R, s, n, masks, window)
    b = dec.new_batch(req, [budget] * n, rules=rules)
    _set_states(b, s, n)
    R.run_ar(dec, b)
    ar = b.transcripts()
    # by hand: one row at a time, the rules on the host
    import speculative_whisper_asr_gb300.binding as B
    stream = torch.cuda.current_stream().cuda_stream
    dec.reset(req)
    scratch = dec.new_batch(req, [10 ** 6] * n)
    hand = [[] for _ in range(n)]
    blk = dev_i32([list(s.prompt)] * n)
    for step in range(budget):
        H = blk.shape[1]
        t, lg = torch.zeros(n, H, dtype=torch.int32, device="cuda"), torch.empty(n, H, s.vocab, device="cuda")
        bl = dev_i32([H] * n)
        dec.verify(req, blk, bl, t, lg)
        a = scratch._args(B.WS_ACCEPT_FORCED, H, blk, bl, t, scratch.block1, scratch.blen)
        B.ws_accept(dec.ctx, n, req.data_ptr(), a, stream)
        z = lg[:, -1:].cpu().numpy()
        hist = np.zeros((n, max(1, step)), np.int32)
        for i in range(n):
            hist[i, :step] = hand[i][:step]
        _, tgt, _ = rules_rule(z, hist, [step] * n, None, None, window, host["rep"], host["pres"], host["freq"], host["bias"],
                               host["masks"], np.arange(n)[:, None])
        for i in range(n):
            hand[i].append(int(tgt[i, 0]))
        blk = dev_i32([[hand[i][-1]] for i in range(n)])
    for i in range(n):
        k = hand[i].index(s.eos_id) + 1 if s.eos_id in hand[i] else budget
        assert ar[i] == hand[i][:k]
    assert any(len(set(x)) > 4 for x in ar)
    plain = dec.new_batch(req, [budget] * n)
    R.run_ar(dec, plain)
    assert plain.transcripts() != ar                          # the rules matter
    for kw in (dict(), dict(graph=False), dict(k_verify=3)):
        sp = dec.new_batch(req, [budget] * n, rules=rules)
        _set_states(sp, s, n)
        if "k_verify" in kw:
            sp.states(4).copy_(torch.arange(n, device="cuda", dtype=torch.int32)[:, None].expand(n, 4))
        R.run_spec(dec, sp, **kw)
        assert sp.transcripts() == ar
    assert dec.status() == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_sampling_under_rules_obeys_the_grammar(R, dtype):
    n, budget = 2, 30
    s, dec, req, _ = _decoder(R, dtype, n)
    host, rules = _rules(R, s, n)
    for spec in (False, True):
        b = dec.new_batch(req, [budget] * n, sampling=True, rules=rules)
        _set_states(b, s, n)
        if spec:
            R.run_spec(dec, b, temperature=1.0, seed=5)
        else:
            R.run_ar_sampling(dec, b, 1.0, 5)
        for i, tr in enumerate(b.transcripts()):
            assert len(tr) == budget or tr[-1] == s.eos_id
            for t in tr:
                assert (int(host["masks"][i, t // 32]) >> (t % 32)) & 1, (spec, i, t)
    assert dec.status() == 0


def test_rules_refuse_tree_rounds(R):
    s, dec, req, _ = _decoder(R, "f32", 1)
    dec.set_tree((-1, 0, 0), (0, 0, 1))
    b = dec.new_batch(req, [8], rules=_rules(R, s, 1)[1])
    b.prefill()
    with pytest.raises(ValueError):
        b.spec_step(1, tree=True)


# ------------------------------------------------------------------ frames
def _verify(dec, s, req, block, lens):
    n, H = len(block), len(block[0])
    t, lg = torch.zeros(n, H, dtype=torch.int32, device="cuda"), torch.full((n, H, s.vocab), 0.0, device="cuda")
    dec.reset(req)
    dec.verify(req, dev_i32(block), dev_i32(lens), t, lg)
    torch.cuda.synchronize()
    return lg.cpu().numpy()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("frames", [(140, 90), (1, 64), (300, 257)])
def test_frame_mass_adds_up(R, dtype, frames):
    """Every row's weights add up to one per layer and head, nothing lands behind the valid frames or on other slots,
    and the logits stay within the model's tolerance."""
    s, dec, req, _ = _decoder(R, dtype, 2, frames)
    g = np.random.default_rng(1)
    block, lens = g.integers(0, s.vocab, (2, 9)).tolist(), [9, 5]
    plain = _verify(dec, s, req, block, lens)
    dec.accumulate_frames(True)
    got = _verify(dec, s, req, block, lens)
    mass = dec.frame_mass().double().cpu()
    for i in range(2):
        logits_close(got[i, : lens[i]], plain[i, : lens[i]], 1e-4 if dtype == "f32" else 2e-2)
        total = mass[:, i].sum(-1)
        # a row's weights sum to 1 within the exponentials' 2^-20 and 300 sums' steps
        assert bool((total - lens[i]).abs().max() < lens[i] * (2.0 ** -19 + 300 * 2.0 ** -24)), total
        assert bool((mass[:, i, :, frames[i]:] == 0).all())
    assert bool((mass >= 0).all())
    dec.accumulate_frames(False)
    again = _verify(dec, s, req, block, lens)
    assert np.array_equal(again, plain)                       # off: the usual path, bit for bit
    assert torch.equal(dec.frame_mass().double().cpu(), mass)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_cut_cache_equals_a_cache_of_the_kept_frames(R, dtype):
    """The same frames kept in every layer and head: as if only they had been encoded."""
    s, dec, req, A = _decoder(R, dtype, 2, (140, 90))
    g = np.random.default_rng(2)
    block, lens = g.integers(0, s.vocab, (2, 9)).tolist(), [9, 9]
    full = _verify(dec, s, req, block, lens)
    keep, sets = 60, [np.sort(g.choice(f, 60, replace=False)) for f in (140, 90)]
    mass = dec.frame_mass()
    for i, k in enumerate(sets):
        mass[:, i, :, torch.as_tensor(k, device="cuda")] = 1.0 + torch.rand(len(k), device="cuda")
    # the drafter reads its own caches: the same proposals before and after
    b = dec.new_batch(req, [20, 20], draft_logits=True)
    b.prefill()
    dec.draft(req, b.block, q_logits=b.q_logits)
    before = b.q_logits.clone()
    dec.evict_frames(req, keep)
    dec.draft(req, b.block, q_logits=b.q_logits)
    assert torch.equal(before, b.q_logits)
    assert bool((dec.frame_mass() == 0).all())
    cut = _verify(dec, s, req, block, lens)
    assert not np.array_equal(cut, full)
    other = R.Decoder(s, synth.target_weights(s, 3), None, max_batch=2, max_frames=140)
    oreq = other.slots([0, 1])
    other.cross_kv(oreq, torch.cat([other.enc_tensor(a[k]) for a, k in zip(A, sets)]), [keep, keep])
    want = _verify(other, s, oreq, block, lens)
    logits_close(cut.reshape(-1, s.vocab), want.reshape(-1, s.vocab), 1e-4 if dtype == "f32" else 2e-2)
    # new acoustic keys give the slots their full caches back
    dec.cross_kv(req, torch.cat([dec.enc_tensor(a) for a in A]), [140, 90])
    assert np.array_equal(_verify(dec, s, req, block, lens), full)


def test_evict_frames_leaves_other_slots_and_short_requests(R):
    s, dec, req, A = _decoder(R, "bf16", 2, (140, 50))
    g = np.random.default_rng(3)
    block = g.integers(0, s.vocab, (2, 4)).tolist()
    full = _verify(dec, s, req, block, [4, 4])
    dec.frame_mass().uniform_()
    dec.evict_frames(dec.slots([1]), 60)                      # already fits
    assert np.array_equal(_verify(dec, s, req, block, [4, 4]), full)
    dec.frame_mass().uniform_()
    dec.evict_frames(req, 50)
    cut = _verify(dec, s, req, block, [4, 4])
    assert np.array_equal(cut[1], full[1]) and not np.array_equal(cut[0], full[0])


def test_evict_frames_refusals(R):
    import speculative_whisper_asr_gb300.binding as B
    s, dec, req, _ = _decoder(R, "f32", 2)
    for keep in (0, 141):
        with pytest.raises(B.WSError) as e:
            dec.evict_frames(req, keep)
        assert e.value.code == B.WS_EINVAL
    dec.set_readout(1, 10)
    with pytest.raises(B.WSError) as e:
        dec.evict_frames(req, 50)
    assert e.value.code == B.WS_EUNSUPPORTED
    dec.set_readout(-1, 0)
    dec.evict_frames(req, 50)
    with pytest.raises(B.WSError) as e:
        dec.set_readout(1, 10)
    assert e.value.code == B.WS_EUNSUPPORTED


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("spec", [False, True])
def test_decoding_with_cut_caches(R, dtype, spec):
    """keep_frames in the loop: keeping every frame changes nothing beyond the kernels' tolerance; cutting runs to the
    end, and the weights of the accumulated rounds are gone afterwards."""
    s, dec, req, A = _decoder(R, dtype, 2, (140, 90))
    run = R.run_spec if spec else R.run_ar
    b = dec.new_batch(req, [30, 30])
    rounds = run(dec, b, keep_frames=40, evict_after=3)
    assert rounds >= 1 and dec.accumulating is False
    for tr in b.transcripts():
        assert len(tr) == 30 or tr[-1] == s.eos_id
    assert bool((dec.frame_mass() == 0).all()) or rounds <= 3
    again = dec.new_batch(req, [30, 30])                      # the caches are cut now: plain decoding over them
    run(dec, again)
    other = dec.new_batch(req, [30, 30])
    (R.run_ar if spec else R.run_spec)(dec, other)
    assert again.transcripts() == other.transcripts()         # speculative equals autoregressive over cut caches too
    assert dec.status() == 0

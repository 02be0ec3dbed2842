"""Host driver for libws: device buffers (PyTorch), weight upload and the
propose / verify / accept loop.  Every step of the decoding path runs in the
library's CUDA kernels; this module only allocates memory, marshals
arguments and decides when the loop stops.

Loop (Whisper-Flash §3.1, Appendix A.1):
  prefill   : ws_verify(prompt) + ws_accept(FORCED) -> first anchor
  each round: ws_draft (or ws_draft_synthetic) -> ws_verify(K+1 rows)
              -> ws_accept (greedy or rejection rule) -> next anchor
  AR greedy : ws_verify(1 row) + ws_accept with no proposals
"""
from __future__ import annotations

from dataclasses import dataclass, field

import numpy as np
import torch

import synth
from . import binding as B


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def _stream():
    return torch.cuda.current_stream().cuda_stream


@dataclass
class RunStats:
    rounds: int = 0
    proposed: int = 0
    accepted: int = 0
    emitted: int = 0
    per_round_acc: list = field(default_factory=list)


class Decoder:
    """One libws context on the current CUDA device."""

    def __init__(self, shape: synth.ModelShape, target: dict, drafter: dict | None, max_batch: int,
                 max_frames: int = 1500, gemm: int = B.WS_GEMM_AUTO, max_block: int | None = None):
        if not torch.cuda.is_available():
            raise RuntimeError("libws needs a CUDA device")
        self.s = shape
        self.dev = torch.device("cuda", torch.cuda.current_device())
        self.max_batch = max_batch
        self.max_frames = max_frames
        self.K = shape.K
        self.V = shape.vocab
        self.dtype = B.WS_BF16 if shape.dtype == "bf16" else B.WS_F32
        self.tdtype = torch.bfloat16 if shape.dtype == "bf16" else torch.float32
        self.readout = False
        self.accumulating = False
        self._mass = None
        self.tree = None
        dl = shape.drafter_layers if drafter is not None else 0
        self.max_block = max_block or max(shape.K + 1, len(shape.prompt))
        self.desc = B.make_desc(shape.n_layers, shape.d_model, shape.n_heads, shape.d_ff, shape.vocab,
                                shape.max_pos, dl, shape.hist_layers, shape.K, self.dtype, max_batch, max_frames,
                                self.max_block, shape.eos_id, gemm)
        nbytes = B.ws_query_workspace(self.desc)
        if nbytes == 0:
            raise ValueError("invalid model description")
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=self.dev)
        tblob = self._blob(target, synth.target_tensor_shapes(shape))
        dblob = self._blob(drafter, synth.drafter_tensor_shapes(shape)) if dl else None
        self.ctx = B.ws_load_weights(self.desc, self.workspace.data_ptr(), nbytes, tblob.data_ptr(),
                                     _ptr(dblob), _stream())
        del tblob, dblob
        self.engine = B.ws_gemm_engine(self.ctx)

    def __del__(self):
        ctx = getattr(self, "ctx", None)
        if ctx:
            B.ws_free(ctx)
            self.ctx = None

    def _blob(self, tensors, order):
        t = torch.from_numpy(synth.blob_from(tensors, order, self.s.dtype))
        if self.s.dtype == "bf16":
            t = t.view(torch.int16)
        return t.to(self.dev)

    def enc_tensor(self, A: np.ndarray) -> torch.Tensor:
        """Encoder states (already in the model's value set) as a device tensor."""
        if self.s.dtype == "bf16":
            return torch.from_numpy(synth.bf16_bits(A)).view(torch.int16).to(self.dev).view(torch.bfloat16)
        return torch.from_numpy(np.ascontiguousarray(A, dtype=np.float32)).to(self.dev)

    # ------------------------------------------------------------------ raw calls
    def slots(self, ids) -> torch.Tensor:
        return torch.as_tensor(np.asarray(ids, dtype=np.int32), device=self.dev)

    def reset(self, req):
        B.ws_reset(self.ctx, req.numel(), req.data_ptr(), _stream())

    def cross_kv(self, req, enc_packed: torch.Tensor, frames, valid=None):
        frames = np.asarray(frames, dtype=np.int32)
        cu = torch.as_tensor(np.concatenate([[0], np.cumsum(frames)]).astype(np.int32), device=self.dev)
        vt = None if valid is None else torch.as_tensor(np.asarray(valid, dtype=np.int32), device=self.dev)
        B.ws_cross_kv(self.ctx, req.numel(), req.data_ptr(), enc_packed.data_ptr(), cu.data_ptr(), _ptr(vt),
                      int(frames.max()), int(frames.sum()), _stream())
        return cu, vt

    def verify(self, req, block, block_len, target, logits=None):
        n, H = block.shape
        B.ws_verify(self.ctx, n, req.data_ptr(), H, block.data_ptr(), block_len.data_ptr(), target.data_ptr(),
                    _ptr(logits), _stream())

    def draft(self, req, block, temperature=0.0, seed=0, rnd=0, q_logits=None):
        B.ws_draft(self.ctx, req.numel(), req.data_ptr(), block.data_ptr(), float(temperature), seed, rnd,
                   _ptr(q_logits), _stream())

    def sample(self, req, logits, temperature, seed, rnd, out):
        n, rows = out.shape
        B.ws_sample(self.ctx, n, req.data_ptr(), logits.data_ptr(), rows, float(temperature), seed, rnd,
                    out.data_ptr(), _stream())

    def lengths(self, req) -> np.ndarray:
        out = torch.empty(req.numel(), dtype=torch.int32, device=self.dev)
        B.ws_get_lengths(self.ctx, req.numel(), req.data_ptr(), out.data_ptr(), _stream())
        return out.cpu().numpy()

    def status(self) -> int:
        return B.ws_status(self.ctx, _stream())

    def set_readout(self, layer: int, half_width: int):
        """Verification-attention readout at `layer` centring a +-half_width
        frame window on the drafter's cross-attention (layer -1: off)."""
        B.ws_set_readout(self.ctx, layer, half_width)
        self.readout = layer >= 0

    def set_tree(self, parent=(), rank=()):
        """Candidate tree of block rows for tree verification (Alignment Drift
        App. E.3): parent[j] < j (parent[0] = -1), rank[j] = which of the
        drafter's ranked tokens row j takes at its depth; empty: no tree."""
        B.ws_set_tree(self.ctx, list(parent), list(rank))
        self.tree = (tuple(parent), tuple(rank)) if len(parent) else None

    def centers(self, req) -> np.ndarray:
        out = torch.empty(req.numel(), dtype=torch.int32, device=self.dev)
        B.ws_get_centers(self.ctx, req.numel(), req.data_ptr(), out.data_ptr(), _stream())
        return out.cpu().numpy()

    def frame_mass(self) -> torch.Tensor:
        """The decoder's accumulated frame weights [layers, slots, heads, frames] (allocated, zero, on first use)."""
        if self._mass is None:
            self._mass = torch.zeros(self.s.n_layers, self.max_batch, self.s.n_heads, self.max_frames, device=self.dev)
        return self._mass

    def accumulate_frames(self, on: bool):
        """Whether verification adds the rows' cross-attention weights to frame_mass() (ws_set_frame_mass)."""
        B.ws_set_frame_mass(self.ctx, self.frame_mass().data_ptr() if on else 0)
        self.accumulating = on

    def evict_frames(self, req, keep: int):
        """Cut the requests' acoustic caches to the `keep` frames of the largest weight per layer and head
        (ws_evict_frames) and clear their masses, whose positions are the caches' no more."""
        mass = self.frame_mass()
        B.ws_evict_frames(self.ctx, req.numel(), req.data_ptr(), mass.data_ptr(), keep, _stream())
        mass.index_fill_(1, req.long(), 0.0)

    # ------------------------------------------------------------------ batch state
    def new_batch(self, req, budgets, tcap: int | None = None, sampling: bool = False,
                  draft_logits: bool = False, rules: "LogitsRules | None" = None, next_states=None) -> "Batch":
        """draft_logits: keep the drafter's logits also for greedy decoding
        (needed by a confidence threshold).  rules: penalties, biases and
        grammar masks applied to the target's logits of every round.
        next_states(batch, block, block_len, states): called in every round
        once the block is known and before the rules read the grammar states;
        it enqueues on the current stream what sets states [n, H].  Column j of
        block [n, H] is the token before row j (column 0 the anchor, the last
        of batch.transcript); for the prompt block is None and the transcript
        empty.  A grammar whose state depends on the tokens needs it, because
        the proposals do not exist before the round; its rounds are not
        replayed from a graph."""
        return Batch(self, req, budgets, tcap or self.s.max_pos, sampling, draft_logits, rules, next_states)


class Batch:
    """Device arrays of one decoding batch (request slots `req`)."""

    def __init__(self, dec: Decoder, req: torch.Tensor, budgets, tcap: int, sampling: bool,
                 draft_logits: bool = False, rules: "LogitsRules | None" = None, next_states=None):
        if next_states is not None and (rules is None or not rules.has_masks):
            raise ValueError("next_states sets grammar states: rules with masks are needed")
        self.dec = dec
        self.req = req
        n = req.numel()
        self.n = n
        dev, K = dec.dev, dec.K
        i32 = dict(dtype=torch.int32, device=dev)
        self.block = torch.zeros(n, K + 1, **i32)
        self.blen = torch.zeros(n, **i32)
        self.target = torch.zeros(n, K + 1, **i32)
        self.block1 = torch.zeros(n, 1, **i32)
        self.target1 = torch.zeros(n, 1, **i32)
        self.prompt = torch.as_tensor(np.tile(np.asarray(dec.s.prompt, dtype=np.int32), (n, 1)), device=dev)
        self.plen = torch.full((n,), len(dec.s.prompt), **i32)
        self.ptarget = torch.zeros(n, len(dec.s.prompt), **i32)
        self.budget = torch.as_tensor(np.asarray(budgets, dtype=np.int32), device=dev).clone()
        self.done = torch.zeros(n, **i32)
        self.n_acc = torch.zeros(n, **i32)
        self.n_emit = torch.zeros(n, **i32)
        self.transcript = torch.full((n, tcap), -1, **i32)
        self.out_len = torch.zeros(n, **i32)
        self.n_done = torch.zeros(1, **i32)
        self.tcap = tcap
        self.acc_sum = torch.zeros(n, dtype=torch.int64, device=dev)
        self.prop_sum = torch.zeros(n, dtype=torch.int64, device=dev)
        self.p_logits = self.q_logits = self.p_logits1 = None
        self.rules = rules
        self.next_states = next_states
        self._states = {}
        if sampling or rules is not None:
            rows = max(K + 1, len(dec.s.prompt)) if rules is not None else K + 1
            self._p_store = torch.empty(n * rows * dec.V, dtype=torch.float32, device=dev)
            self.p_logits = self._p_store[: n * (K + 1) * dec.V].view(n, K + 1, dec.V)
        if sampling or draft_logits or dec.tree is not None:
            self.q_logits = torch.empty(n, K, dec.V, dtype=torch.float32, device=dev)
        self.vblock = torch.zeros(n, K + 1, **i32)      # the block as verified (truncated proposals)
        self.tblock = torch.zeros(n, dec.max_block, **i32)    # a candidate tree's tokens
        self.ttarget = torch.zeros(n, dec.max_block, **i32)
        self.host_done = torch.zeros(1, dtype=torch.int32).pin_memory()
        self.graphs = {}

    def __del__(self):
        for g in getattr(self, "graphs", {}).values():
            B.ws_graph_free(g)

    def replay(self, key, fn):
        """Run `fn` (a fixed sequence of ws_* calls) through a CUDA graph
        captured on first use; later calls replay it."""
        g = self.graphs.get(key)
        s = _stream()
        if g is None:
            B.ws_capture_begin(self.dec.ctx, s)
            try:
                fn()
            finally:
                g = B.ws_capture_end(self.dec.ctx, s)
            self.graphs[key] = g
        B.ws_graph_launch(g, s)

    def _logits(self, H):
        """The target logits of an H-row verify, [n, H, vocab]."""
        return self._p_store[: self.n * H * self.dec.V].view(self.n, H, self.dec.V)

    def states(self, H: int) -> torch.Tensor:
        """Grammar states [n, H] int32 of the rows of H-row blocks (a prompt, a single token, a verified block: row j
        follows the block's first j proposals), read by every round of that height; -1, the start: no constraint.
        They stay as the caller sets them, for grammars with one state per request, unless the batch has
        next_states."""
        if H not in self._states:
            self._states[H] = torch.full((self.n, H), -1, dtype=torch.int32, device=self.dec.dev)
        return self._states[H]

    def _apply_rules(self, H, block, blen, target, prompt=False):
        """The rules on an H-row verify's logits, in place, and the greedy choice under them into target.  The rows
        of a prompt follow no proposals."""
        if self.next_states is not None:
            self.next_states(self, None if prompt else block, blen, self.states(H))
        self.rules.apply(self._logits(H), history=self.transcript, hist_len=self.out_len,
                         block=None if prompt else block, block_len=blen,
                         mask_row=self.states(H) if self.rules.has_masks else None,
                         target=target.view(-1)[: self.n * H].view(self.n, H))

    def _args(self, mode, H, block, blen, target, next_block, next_len, p_logits=None, q_logits=None,
              temperature=0.0, seed=0, rnd=0) -> B.AcceptArgs:
        a = B.AcceptArgs()
        a.mode, a.H = mode, H
        a.block, a.block_len, a.target = block.data_ptr(), blen.data_ptr(), _ptr(target)
        a.p_logits, a.q_logits = _ptr(p_logits), _ptr(q_logits)
        a.temperature, a.seed, a.round = float(temperature), int(seed), int(rnd)
        a.budget, a.done, a.n_acc, a.n_emit = (self.budget.data_ptr(), self.done.data_ptr(),
                                               self.n_acc.data_ptr(), self.n_emit.data_ptr())
        a.next_block, a.next_stride, a.next_len = next_block.data_ptr(), next_block.shape[1], next_len.data_ptr()
        a.transcript, a.out_len, a.tcap = self.transcript.data_ptr(), self.out_len.data_ptr(), self.tcap
        a.n_done = self.n_done.data_ptr()
        return a

    def prefill(self, ar: bool = False, temperature: float = 0.0, seed: int = 0):
        """Prompt pass: emits the first transcript token (the first anchor)."""
        d = self.dec
        d.reset(self.req)
        sampled = temperature > 0.0 and self.p_logits is not None
        P = self.prompt.shape[1]
        d.verify(self.req, self.prompt, self.plen, self.ptarget,
                 self._logits(P) if self.rules is not None else self.p_logits if sampled else None)
        if self.rules is not None:
            self._apply_rules(P, self.prompt, self.plen, self.ptarget, prompt=True)
        nb = self.block1 if ar else self.block
        a = self._args(B.WS_ACCEPT_FORCED, self.prompt.shape[1], self.prompt, self.plen, self.ptarget, nb,
                       self.blen, self.p_logits if sampled else None, None, temperature if sampled else 0.0,
                       seed, 0)
        B.ws_accept(d.ctx, self.n, self.req.data_ptr(), a, _stream())
        if d.readout and not ar:
            B.ws_readout(d.ctx, self.n, self.req.data_ptr(), self.n_acc.data_ptr(), _stream())

    def ar_step(self, graph: bool = True):
        d = self.dec

        def calls():
            d.verify(self.req, self.block1, self.blen, self.target1,
                     self._logits(1) if self.rules is not None else None)
            if self.rules is not None:
                self._apply_rules(1, self.block1, self.blen, self.target1)
            a = self._args(B.WS_ACCEPT_GREEDY, 1, self.block1, self.blen, self.target1, self.block1, self.blen)
            B.ws_accept(d.ctx, self.n, self.req.data_ptr(), a, _stream())
        self.states(1)                     # allocated outside the capture
        if graph and self.next_states is None:
            self.replay(("ar", d.accumulating), calls)
        else:
            calls()

    def ar_sample_step(self, rnd: int, temperature: float, seed: int):
        """Autoregressive sampling round: verify the anchor, draw from softmax(z/T)."""
        d = self.dec
        d.verify(self.req, self.block1, self.blen, self.target1,
                 self._logits(1) if self.rules is not None else self.p_logits)
        if self.rules is not None:
            self._apply_rules(1, self.block1, self.blen, self.target1)
        a = self._args(B.WS_ACCEPT_SAMPLE, 1, self.block1, self.blen, self.target1, self.block1, self.blen,
                       self.p_logits, self.q_logits, temperature, seed, rnd)
        B.ws_accept(d.ctx, self.n, self.req.data_ptr(), a, _stream())

    def spec_step(self, rnd: int, synthetic=None, temperature: float = 0.0, seed: int = 0, run_drafter=True,
                  graph: bool = True, k_verify: int | None = None, threshold: float = 0.0, tree: bool = False):
        """One propose / verify / accept round.  `synthetic` = (traj, cmask, ctok) device tensors.
        k_verify / threshold: verify only the first k_verify proposals, stopping
        before the first one whose drafter confidence is below threshold
        (ws_draft_limit).  Greedy rounds replay one captured graph per
        (proposal source, verify length, threshold): their calls do not depend
        on the round.  tree: the drafter's ranked tokens fill the decoder's
        candidate tree (set_tree), verified in one pass and accepted along
        the longest matching root path (greedy only)."""
        self.states(self.dec.K + 1 if k_verify is None else k_verify + 1)     # allocated outside a capture
        self.states(self.dec.K + 1)
        if tree:
            if temperature > 0.0 or synthetic is not None or not run_drafter or self.dec.tree is None:
                raise ValueError("tree rounds need set_tree, the drafter and greedy decoding")
            if self.rules is not None:
                raise ValueError("logits rules follow linear blocks: not in tree rounds")
            if graph:
                self.replay(("tree", self.dec.tree, self.dec.accumulating), self._tree_calls)
            else:
                self._tree_calls()
        elif graph and temperature <= 0.0 and self.next_states is None:
            self.replay(("spec", synthetic is not None, run_drafter, k_verify, threshold, self.dec.accumulating),
                        lambda: self._spec_calls(0, synthetic, 0.0, 0, run_drafter, k_verify, threshold))
        else:
            self._spec_calls(rnd, synthetic, temperature, seed, run_drafter, k_verify, threshold)

    def _tree_calls(self):
        d = self.dec
        N = len(d.tree[0])
        req = self.req.data_ptr()
        d.draft(self.req, self.block, 0.0, 0, 0, self.q_logits)
        B.ws_tree_tokens(d.ctx, self.n, req, self.block.data_ptr(), d.K + 1, self.q_logits.data_ptr(),
                         self.tblock.data_ptr(), N, self.blen.data_ptr(), _stream())
        B.ws_verify_tree(d.ctx, self.n, req, N, self.tblock.data_ptr(), self.blen.data_ptr(),
                         self.ttarget.data_ptr(), 0, _stream())
        a = self._args(B.WS_ACCEPT_TREE, N, self.tblock, self.blen, self.ttarget, self.block, self.blen)
        B.ws_accept(d.ctx, self.n, req, a, _stream())
        if d.readout:              # the path's rows are in block order after acceptance
            B.ws_readout(d.ctx, self.n, req, self.n_acc.data_ptr(), _stream())

    def _spec_calls(self, rnd, synthetic, temperature, seed, run_drafter, k_verify=None, threshold=0.0):
        d = self.dec
        sampling = temperature > 0.0
        K = d.K
        limited = k_verify is not None and (k_verify < K or threshold > 0.0)
        if run_drafter:
            d.draft(self.req, self.block, temperature, seed, rnd,
                    self.q_logits if (sampling or threshold > 0.0) else None)
        if synthetic is not None:
            traj, cmask, ctok = synthetic
            B.ws_draft_synthetic(d.ctx, self.n, self.req.data_ptr(), self.block.data_ptr(), traj.data_ptr(),
                                 traj.shape[1], cmask.data_ptr(), ctok.data_ptr(), _stream())
        H, vb = K + 1, self.block
        if limited:
            H, vb = k_verify + 1, self.vblock
            B.ws_draft_limit(d.ctx, self.n, self.req.data_ptr(), self.block.data_ptr(), K + 1,
                             _ptr(self.q_logits) if threshold > 0.0 else 0, k_verify, threshold, temperature,
                             vb.data_ptr(), H, self.blen.data_ptr(), _stream())
        B.ws_verify(d.ctx, self.n, self.req.data_ptr(), H, vb.data_ptr(), self.blen.data_ptr(),
                    self.target.data_ptr(),
                    self._logits(H).data_ptr() if self.rules is not None else _ptr(self.p_logits) if sampling else 0,
                    _stream())
        if self.rules is not None:
            self._apply_rules(H, vb.view(-1)[: self.n * H].view(self.n, H), self.blen, self.target)
        mode = B.WS_ACCEPT_SAMPLE if sampling else B.WS_ACCEPT_GREEDY
        a = self._args(mode, H, vb, self.blen, self.target, self.block, self.blen,
                       self.p_logits, self.q_logits, temperature, seed, rnd)
        B.ws_accept(d.ctx, self.n, self.req.data_ptr(), a, _stream())
        if d.readout:              # the row that produced the next anchor centres the next draft window
            B.ws_readout(d.ctx, self.n, self.req.data_ptr(), self.n_acc.data_ptr(), _stream())

    def poll_done(self) -> int:
        self.host_done.copy_(self.n_done, non_blocking=True)
        torch.cuda.current_stream().synchronize()
        return int(self.host_done.item())

    def transcripts(self):
        t = self.transcript.cpu().numpy()
        n = self.out_len.cpu().numpy()
        return [list(map(int, t[i, :n[i]])) for i in range(self.n)]


def _frames_round(dec: Decoder, batch: Batch, rounds: int, keep_frames, evict_after: int):
    """Before round `rounds` (0: the prompt): frame weights are accumulated up to round `evict_after`, after which
    the caches are cut to keep_frames."""
    if keep_frames is None or rounds > evict_after:
        return
    if rounds == 0:
        dec.frame_mass().index_fill_(1, batch.req.long(), 0.0)
        dec.accumulate_frames(True)
    if rounds == evict_after:
        dec.accumulate_frames(False)
        dec.evict_frames(batch.req, keep_frames)


def run_ar(dec: Decoder, batch: Batch, max_rounds: int = 100000, keep_frames: int | None = None,
           evict_after: int = 8) -> int:
    """keep_frames: after `evict_after` rounds keep only that many acoustic frames per layer and head, those with the
    most attention so far (approximate)."""
    rounds = 0
    try:
        _frames_round(dec, batch, 0, keep_frames, max(1, evict_after))
        batch.prefill(ar=True)
        while batch.poll_done() < batch.n and rounds < max_rounds:
            if rounds:
                _frames_round(dec, batch, rounds, keep_frames, max(1, evict_after))
            batch.ar_step()
            rounds += 1
    finally:
        if dec.accumulating and keep_frames is not None:
            dec.accumulate_frames(False)
    return rounds


def run_spec(dec: Decoder, batch: Batch, synthetic=None, temperature=0.0, seed=0, max_rounds=100000,
             run_drafter=True, graph=True, k_verify=None, threshold=0.0, tree=False, keep_frames: int | None = None,
             evict_after: int = 8) -> int:
    """keep_frames, evict_after: as for run_ar."""
    rounds = 0
    try:
        _frames_round(dec, batch, 0, keep_frames, max(1, evict_after))
        batch.prefill(temperature=temperature, seed=seed)
        while batch.poll_done() < batch.n and rounds < max_rounds:
            if rounds:
                _frames_round(dec, batch, rounds, keep_frames, max(1, evict_after))
            batch.spec_step(rounds + 1, synthetic, temperature, seed, run_drafter, graph=graph, k_verify=k_verify,
                            threshold=threshold, tree=tree)
            rounds += 1
    finally:
        if dec.accumulating and keep_frames is not None:
            dec.accumulate_frames(False)
    return rounds


def run_ar_sampling(dec: Decoder, batch: Batch, temperature: float, seed: int, max_rounds=100000) -> int:
    batch.prefill(ar=True, temperature=temperature, seed=seed)
    rounds = 0
    while batch.poll_done() < batch.n and rounds < max_rounds:
        rounds += 1
        batch.ar_sample_step(rounds, temperature, seed)
    return rounds


def run_spec_packed(dec: Decoder, req_all: torch.Tensor, budgets, synthetic=None, max_rounds=100000,
                    live_rounds: list | None = None):
    """Varlen batch without padding rows: after every round the requests that
    finished are dropped from the slot list, so later rounds only carry live
    requests (their rows, attention and acceptance).  Returns (transcripts,
    rounds, rows processed); `live_rounds`, when given, receives the number
    of rounds each request took part in."""
    n_all = req_all.numel()
    alive = list(range(n_all))
    out = [None] * n_all
    live = [0] * n_all
    budgets = np.asarray(budgets, dtype=np.int32)
    b = dec.new_batch(req_all, budgets)
    b.prefill()
    rounds, rows = 0, 0
    syn_all = synthetic
    while rounds < max_rounds:
        done = b.done.cpu().numpy()
        if done.any():
            tr = b.transcripts()
            keep = [k for k in range(len(alive)) if not done[k]]
            for k in range(len(alive)):
                if done[k]:
                    out[alive[k]] = tr[k]
            if not keep:
                break
            idx = torch.as_tensor(keep, device=dec.dev, dtype=torch.long)
            nb = dec.new_batch(b.req[idx].contiguous(), b.budget[idx].cpu().numpy(), b.tcap)
            for name in ("block", "blen", "budget", "done", "out_len", "transcript"):
                getattr(nb, name).copy_(getattr(b, name)[idx])
            if syn_all is not None:
                syn_all = tuple(t[idx].contiguous() for t in syn_all)
            alive = [alive[k] for k in keep]
            b = nb
        rounds += 1
        rows += b.n * (dec.K + 1)
        for k in alive:
            live[k] += 1
        b.spec_step(rounds, syn_all, graph=False)
    if live_rounds is not None:
        live_rounds[:] = live
    return out, rounds, rows


class Encoder:
    """libws audio encoder on the current CUDA device (bf16): log-mel windows
    [n, n_mels, 2F] -> encoder states [n, F, d], the input of Decoder.cross_kv."""

    def __init__(self, shape: synth.EncoderShape, weights: dict, max_batch: int):
        if not torch.cuda.is_available():
            raise RuntimeError("libws needs a CUDA device")
        if shape.dtype != "bf16":
            raise ValueError("the encoder runs in bf16")
        self.s = shape
        self.dev = torch.device("cuda", torch.cuda.current_device())
        self.max_batch = max_batch
        self.desc = B.make_encoder_desc(shape.n_layers, shape.d_model, shape.n_heads, shape.d_ff, shape.n_mels,
                                        shape.n_frames, max_batch)
        nbytes = B.ws_encoder_workspace(self.desc)
        if nbytes == 0:
            raise ValueError("invalid encoder description")
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=self.dev)
        blob = torch.from_numpy(synth.blob_from(weights, synth.encoder_tensor_shapes(shape), "bf16"))
        blob = blob.view(torch.int16).to(self.dev)
        self.enc = B.ws_encoder_load(self.desc, self.workspace.data_ptr(), nbytes, blob.data_ptr(), _stream())
        del blob

    def __del__(self):
        enc = getattr(self, "enc", None)
        if enc:
            B.ws_encoder_free(enc)
            self.enc = None

    def mel_tensor(self, mels) -> torch.Tensor:
        """Stack bf16-valued log-mel arrays [n_mels, 2F] into one device tensor."""
        a = np.stack([np.asarray(m, dtype=np.float32) for m in mels])
        return torch.from_numpy(synth.bf16_bits(a)).view(torch.int16).to(self.dev).view(torch.bfloat16)

    def encode(self, mel: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
        n = mel.shape[0]
        if out is None:
            out = torch.empty(n, self.s.n_frames, self.s.d_model, dtype=torch.bfloat16, device=self.dev)
        B.ws_encode(self.enc, n, mel.data_ptr(), out.data_ptr(), _stream())
        return out

    def status(self) -> int:
        return B.ws_encoder_status(self.enc, _stream())

    def set_attention(self, tcgen05: bool):
        """Attention kernel: tcgen05 flash attention (default) or the legacy mma.sync one."""
        B.ws_encoder_attention(self.enc, 1 if tcgen05 else 0)


# ---------------------------------------------------------------------- operators on the caller's tensors
_I32, _F32 = torch.int32, torch.float32


def _rows(name, t, dtype, shape, dev):
    """Pointer of a contiguous tensor of exactly this type and shape on CUDA device number `dev`."""
    if t is None or t.dtype is not dtype or t.get_device() != dev or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{dev} is needed")
    return t.data_ptr()


def _per_position(name, t, dtype, slots, heads, dev):
    """Pointer and width of a contiguous [slots, heads, width] tensor."""
    s = t.shape
    if (t.dtype is not dtype or t.get_device() != dev or len(s) != 3 or s[0] != slots or s[1] != heads
            or not t.is_contiguous()):
        raise ValueError(f"{name}: a contiguous {dtype} tensor [{slots}, {heads}, width] on cuda:{dev} is needed")
    return t.data_ptr(), s[2]


def _on(dev):
    """The handle of the current stream; device number `dev` has to be the current device."""
    if torch.cuda.current_device() != dev:
        raise ValueError(f"the tensors are on cuda:{dev}, the current device is cuda:{torch.cuda.current_device()}")
    return torch._C._cuda_getCurrentRawStream(dev)


class PagedCache:
    """A paged key/value cache in the caller's tensors (ws_paged_cache):
    k, v [pages, KV heads, page_size, 64] with any strides that are multiples
    of 16 bytes (the same for both), page_table [slots, pages per slot] int32.
    The object keeps scratch for each stream that called it; graphs captured
    on one stream share it with each other and with calls on that stream, so
    what may run at the same time needs a PagedCache each.  One thread at a
    time calls it."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, page_table: torch.Tensor):
        if k.dtype not in (torch.bfloat16, torch.float32) or k.dim() != 4 or k.shape[3] != 64 or not k.is_cuda:
            raise ValueError("k: a CUDA tensor [pages, heads, page_size, 64] in bf16 or fp32 is needed")
        if v.dtype is not k.dtype or v.shape != k.shape or v.stride() != k.stride() or v.device != k.device:
            raise ValueError("v must have the type, shape, strides and device of k")
        if k.stride(3) != 1:
            raise ValueError("the head dimension must be contiguous")
        if (page_table.dtype is not _I32 or page_table.dim() != 2 or page_table.device != k.device
                or not page_table.is_contiguous()):
            raise ValueError("page_table: a contiguous int32 tensor [slots, pages] on k's device is needed")
        self.k, self.v, self.page_table = k, v, page_table
        self.dev, self.dtype = k.get_device(), k.dtype
        self.pages, self.heads, self.page_size, _ = k.shape
        self.slots = page_table.shape[0]
        self.desc = B.PagedCacheDesc(
            B.WS_BF16 if k.dtype is torch.bfloat16 else B.WS_F32, self.heads, self.page_size, self.pages, k.data_ptr(),
            v.data_ptr(), k.stride(0), k.stride(1), k.stride(2), page_table.data_ptr(), self.slots, page_table.shape[1])
        self._attn, self._evict = B.AttentionArgs(), B.EvictArgs()
        self._ws, self._kept = {}, []      # (pointer, bytes) by stream; the tensors behind them

    def _run(self, call, size, args, stream):
        """The call with this stream's scratch, which grows when the call finds it too small.  Outgrown scratch is kept:
        work in flight or a captured graph may still use it."""
        ptr, nbytes = self._ws.get(stream, (0, 0))
        if nbytes:
            try:
                return call(self.desc, args, ptr, nbytes, stream)
            except B.WSError as e:
                if e.code != B.WS_ENOSPACE:
                    raise
        need = size(self.desc, args)
        if need:
            nbytes = max(need, 2 * nbytes)
            self._kept.append(torch.empty(nbytes, dtype=torch.uint8, device=self.k.device))
            ptr = self._kept[-1].data_ptr()
            self._ws[stream] = ptr, nbytes
        return call(self.desc, args, ptr, nbytes, stream)

    def attend(self, q, kv_len, cu_q, max_q: int, max_kv: int, causal: bool = True, scale: float = 0.125, out=None,
               lse=None, mass=None, req_ids=None):
        """Attention of the chunks q [total_q, heads, 64] over the cache (ws_paged_attention).  kv_len [slots] int32
        counts the chunk's own positions; cu_q [requests + 1] int32.  lse [total_q, heads] fp32 receives the
        log-sum-exp; mass [slots, KV heads, >= max_kv] fp32 is added to.  Returns out."""
        if out is None:
            out = torch.zeros_like(q, memory_format=torch.contiguous_format)
        dev = self.dev
        if q.dim() != 3 or out.shape != q.shape or q.shape[2] != 64:
            raise ValueError("q and out: [rows, heads, 64] are needed")
        rows, heads, _ = q.shape
        a = self._attn
        for name, t in (("q", q), ("out", out)):
            s0, s1, s2 = t.stride()
            if t.dtype is not self.dtype or t.get_device() != dev or s2 != 1 or (heads > 1 and s1 != 64):
                raise ValueError(f"{name}: a {self.dtype} tensor with contiguous heads on cuda:{dev} is needed")
            if rows < 2:
                s0 = heads * 64
            if name == "q":
                a.q, a.q_stride = t.data_ptr(), s0
            else:
                a.out, a.out_stride = t.data_ptr(), s0
        n = cu_q.shape[0] - 1
        a.n_req = n
        a.req_ids = 0 if req_ids is None else _rows("req_ids", req_ids, _I32, (n,), dev)
        a.kv_len = _rows("kv_len", kv_len, _I32, (self.slots,), dev)
        a.cu_q = _rows("cu_q", cu_q, _I32, (n + 1,), dev)
        a.total_q, a.max_q, a.max_kv, a.n_heads, a.causal, a.scale = rows, max_q, max_kv, heads, int(causal), scale
        a.lse = 0 if lse is None else _rows("lse", lse, _F32, (rows, heads), dev)
        if mass is None:
            a.mass = 0
        else:
            a.mass, a.mass_stride = _per_position("mass", mass, _F32, self.slots, self.heads, dev)
        self._run(B.ws_paged_attention, B.ws_paged_attention_workspace, a, _on(dev))
        return out

    def evict(self, kv_len, mass, keep: int, max_kv: int, sink: int = 0, recent: int = 0, page_table_out=None,
              kv_len_out=None, mass_out=None, pos=None, pos_out=None, req_ids=None):
        """Keep min(kv_len, keep) positions per slot and head (ws_cache_evict): the first `sink`, the last `recent`,
        then those of the largest mass.  Without page_table_out the cache, and without kv_len_out / mass_out / pos_out
        the lengths, masses and labels, are compacted in place."""
        a, dev, slots, heads = self._evict, self.dev, self.slots, self.heads
        n = slots if req_ids is None else req_ids.shape[0]
        a.n_req = n
        a.req_ids = 0 if req_ids is None else _rows("req_ids", req_ids, _I32, (n,), dev)
        length = _rows("kv_len", kv_len, _I32, (slots,), dev)
        a.kv_len = length
        a.kv_len_out = length if kv_len_out is None else _rows("kv_len_out", kv_len_out, _I32, (slots,), dev)
        a.max_kv, a.keep, a.sink, a.recent = max_kv, keep, sink, recent
        ptr = _per_position("mass", mass, _F32, slots, heads, dev)
        a.mass, a.mass_stride = ptr
        a.mass_out, a.mass_out_stride = (ptr if mass_out is None
                                         else _per_position("mass_out", mass_out, _F32, slots, heads, dev))
        ptr = (0, 0) if pos is None else _per_position("pos", pos, _I32, slots, heads, dev)
        a.pos, a.pos_stride = ptr
        a.pos_out, a.pos_out_stride = ptr if pos_out is None else _per_position("pos_out", pos_out, _I32, slots, heads, dev)
        if page_table_out is None:
            a.page_table_out = 0
        else:
            a.table_out_stride = width = page_table_out.shape[1]
            a.page_table_out = _rows("page_table_out", page_table_out, _I32, (slots, width), dev)
        self._run(B.ws_cache_evict, B.ws_cache_evict_workspace, a, _on(dev))


class LogitsRules:
    """Penalties, biases and grammar masks of a batch of requests
    (ws_logits_rules).  repetition / presence / frequency: [n] fp32; bias_ids
    [n, entries] int32 with bias_vals and bias_len [n]; masks [states,
    ceil(vocab / 32)] int32 words, bit set = token allowed; window: how many
    of the latest tokens count (0: all).  The tensors stay the object's; their
    contents may change between calls."""

    def __init__(self, repetition=None, presence=None, frequency=None, window: int = 0, bias_ids=None, bias_vals=None,
                 bias_len=None, masks=None):
        self._own = (repetition, presence, frequency, bias_ids, bias_vals, bias_len, masks)
        self.has_masks = masks is not None
        self._args = B.RulesArgs()
        self._args.window = window
        self._shape = None                 # (n, vocab, device) that the object's tensors were checked for

    def _bind(self, n, V, dev):
        a = self._args
        self._shape = None                 # a refusal below leaves the arguments half set
        rep, pres, freq, ids, vals, lens, masks = self._own
        for name, t in (("repetition", rep), ("presence", pres), ("frequency", freq)):
            setattr(a, name, 0 if t is None else _rows(name, t, _F32, (n,), dev))
        a.bias_ids = a.bias_vals = a.bias_len = a.bias_stride = a.masks = a.n_masks = 0
        if ids is not None:
            width = a.bias_stride = ids.shape[1]
            a.bias_ids = _rows("bias_ids", ids, _I32, (n, width), dev)
            a.bias_vals = _rows("bias_vals", vals, _F32, (n, width), dev)
            a.bias_len = _rows("bias_len", lens, _I32, (n,), dev)
        if masks is not None:
            a.n_masks = masks.shape[0]
            a.masks = _rows("masks", masks, _I32, (a.n_masks, (V + 31) // 32), dev)
        self._shape = (n, V, dev)

    def apply(self, logits, history=None, hist_len=None, block=None, block_len=None, mask_row=None, out=None,
              target=None, logprob=None):
        """New logits of rows [n, H, vocab] fp32 into out (default: in place).  history [n, tokens] with hist_len [n]:
        the tokens so far, the anchor included; block [n, >= H]: the block, whose columns 1..j precede row j;
        mask_row [n, H]: each row's grammar state (needed when the object has masks).  target [n, H] int32 and
        logprob [n, H] fp32 receive the greedy choice.  Returns out."""
        out = logits if out is None else out
        dev = logits.get_device()
        n, H, V = logits.shape
        a = self._args
        for t in (logits, out):
            if t.dtype is not _F32 or t.get_device() != dev or dev < 0 or t.shape != logits.shape:
                raise ValueError("logits and out: fp32 CUDA tensors [n, H, vocab] are needed")
            s0, s1, s2 = t.stride()
            ld = s1 if H > 1 else s0 if n > 1 else V
            if (V > 1 and s2 != 1) or (n > 1 and s0 != H * ld):
                raise ValueError("logits and out: evenly spaced contiguous rows are needed")
            if t is logits:
                a.logits, a.ld = t.data_ptr(), ld
            if t is out:
                a.out, a.ld_out = t.data_ptr(), ld
        if self._shape != (n, V, dev):
            self._bind(n, V, dev)
        a.n, a.H, a.vocab = n, H, V
        a.block_len = 0 if block_len is None else _rows("block_len", block_len, _I32, (n,), dev)
        if history is None:
            a.history = 0
        else:
            a.hist_stride = width = history.shape[1]
            a.history = _rows("history", history, _I32, (n, width), dev)
            a.hist_len = _rows("hist_len", hist_len, _I32, (n,), dev)
        if block is None:
            a.block = 0
        else:
            a.block_stride = width = block.shape[1]
            a.block = _rows("block", block, _I32, (n, width), dev)
        a.mask_row = 0 if mask_row is None else _rows("mask_row", mask_row, _I32, (n, H), dev)
        a.target = 0 if target is None else _rows("target", target, _I32, (n, H), dev)
        a.logprob = 0 if logprob is None else _rows("logprob", logprob, _F32, (n, H), dev)
        B.ws_logits_rules(a, _on(dev))
        return out

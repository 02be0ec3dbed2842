"""Refusals of the beam selection where arrays share elements, and the parts that
its rows are cut into (no GPU needed)."""
import pytest

from test_beam_operators_host import B, _beam, _refused  # noqa: F401  (B: the fixture)

M = 1 << 20                                # _beam's arrays are this far apart, but parent and token at 4096 and 8192


@pytest.mark.parametrize("bad", [dict(token=4096), dict(token=4096 + 56), dict(parent=M), dict(token=2 * M + 8), dict(parent=2 * M),
                                 dict(done_score=4096), dict(done_score=2 * M + 56), dict(done_length=9 * M), dict(done_length=9 * M + 56),
                                 dict(done_score=M + 4), dict(parent=3 * M + 26876), dict(token=4 * M), dict(token=5 * M),
                                 dict(done_length=6 * M + 8), dict(length_out=8 * M), dict(n_done_out=5 * M), dict(score_out=9 * M),
                                 dict(token=11 * M + 26876), dict(done_tokens=4096 - 4), dict(tokens_out=11 * M + 4), dict(parent=7 * M - 56),
                                 dict(score_out=3 * M), dict(done_tokens=10 * M), dict(parent=8 * M)])
def test_beam_outputs_that_share_elements_refused(B, bad):
    a = _beam(B, **bad)
    need = B.ws_beam_select_workspace(_beam(B))
    _refused(B, lambda: B.ws_beam_select(a, 1 << 30, need, 0), B.WS_EINVAL)
    assert "share" in B.ws_last_error()


@pytest.mark.parametrize("ok", [dict(), dict(score_out=M, tokens_out=3 * M, length_out=5 * M, n_done_out=7 * M), dict(token=4096 + 60),
                                dict(parent=2 * M - 60), dict(done_score=9 * M, done_length=9 * M + 60, done_tokens=9 * M + 120),
                                dict(parent=2 * M + 60, token=2 * M + 120), dict(max_done=0, done_score=2 * M + 8, done_length=4096)])
def test_beam_outputs_beside_each_other_pass(B, ok):
    """What passes the checks ends at the missing GPU, in a process of its own."""
    import os
    import subprocess
    import sys

    import __graft_entry__ as g
    code = (f"import sys; sys.path[:0] = [{os.path.join(g.ROOT, 'tests')!r}, {g.ROOT!r}]\n"
            "from speculative_whisper_asr_gb300 import binding as B\n"
            "import ctypes as C\n"
            "from test_beam_operators_host import _beam\n"
            f"a = _beam(B, **{ok!r})\n"
            "rc = B.lib.ws_beam_select(C.addressof(a), 1 << 30, 1 << 20, None)\n"
            "assert rc == B.WS_ECUDA, (rc, B.ws_last_error())\n")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300, env=dict(os.environ, CUDA_VISIBLE_DEVICES=""))
    assert r.returncode == 0, r.stderr[-800:]


@pytest.mark.parametrize("n,beams", [(1, 1), (16, 5), (20, 5), (24, 5), (32, 5), (60, 5), (72, 5), (95, 5), (96, 5), (32, 12), (33, 4)])
@pytest.mark.parametrize("vocab", [700, 20000, 51866])
def test_beam_parts_run_at_once(B, n, beams, vocab):
    """The parts of all rows, each a CTA, are no more than ten per SM, what the kernel's registers allow, unless a row
    needs that many; the workspace has beams + 1 candidates and a pair of sums of each."""
    bare = {k: 0 for k in ("tokens", "tokens_out", "length", "length_out", "n_done", "n_done_out", "done_score", "done_length", "done_tokens")}
    need = B.ws_beam_select_workspace(_beam(B, n=n, beams=beams, vocab=vocab, ld=vocab, eos_id=-1, **bare))
    rows = n * beams
    parts = need // (rows * (beams + 2) * 8)
    assert need == -(-rows * parts * (beams + 2) * 8 // 256) * 256
    assert parts >= 1 and (rows * parts <= 10 * 152 or parts == -(-vocab // 32768))

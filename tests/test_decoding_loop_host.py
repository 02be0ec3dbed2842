"""The decoding loops' own state when a round fails (stand-ins for the decoder
and the batch; no GPU needed)."""
import pytest
import torch


class _Decoder:
    def __init__(self):
        self.accumulating = False
        self.mass = torch.zeros(1, 2, 1, 4)

    def frame_mass(self):
        return self.mass

    def accumulate_frames(self, on):
        self.accumulating = on

    def evict_frames(self, req, keep):
        raise RuntimeError("eviction")


class _Batch:
    def __init__(self, fails_at):
        self.req, self.n, self.fails_at, self.rounds = torch.zeros(1, dtype=torch.int32), 1, fails_at, 0

    def prefill(self, **kw):
        if self.fails_at == "prefill":
            raise RuntimeError("prefill")

    def poll_done(self):
        return 0

    def _round(self, *a, **kw):
        self.rounds += 1
        if self.rounds == self.fails_at:
            raise RuntimeError("round")

    ar_step = spec_step = _round


@pytest.fixture(scope="module")
def R():
    import __graft_entry__ as g
    g.build()
    from speculative_whisper_asr_gb300 import runtime
    return runtime


@pytest.mark.parametrize("loop", ["run_ar", "run_spec"])
@pytest.mark.parametrize("fails_at", ["prefill", 1, 3, "evict"])
def test_a_failing_round_ends_the_accumulation(R, loop, fails_at):
    dec, batch = _Decoder(), _Batch(fails_at)
    with pytest.raises(RuntimeError):
        getattr(R, loop)(dec, batch, keep_frames=2, evict_after=4)
    assert dec.accumulating is False


@pytest.mark.parametrize("loop", ["run_ar", "run_spec"])
def test_a_loop_without_eviction_leaves_the_accumulation_on(R, loop):
    """Accumulation that the caller switched on is the caller's."""
    dec = _Decoder()
    dec.accumulating = True
    with pytest.raises(RuntimeError):
        getattr(R, loop)(dec, _Batch(2))
    assert dec.accumulating is True

"""clip_gradients on the host (no GPU): what it hands to the library, with the
launch replaced by a record of it."""
import numpy as np
import pytest

from gradient_reduction_amd import clip, executor
from synth import workloads as wl

SIZES = [64, 5, 33]


def made(**kw):
    w = wl.custom_flush("clip", 2, wl.DT_F32, SIZES, capacity=9000, pre_div=1, value_seed=3)
    return w, executor.from_workload(w, device="cpu", **kw)


@pytest.fixture
def launched(monkeypatch):
    seen = []
    monkeypatch.setattr(clip, "clip_records", lambda recs, *rest: seen.append(recs.copy()))
    return seen


@pytest.mark.parametrize("zero2", [False, True])
def test_a_map_that_was_only_recorded_is_refused(launched, zero2):
    """A recording sets map_built and builds nothing: rows taken from what lies in
    the buffers would be anywhere.  The refusal keeps nothing of it."""
    w, ex = made(reduce_to_owner=not zero2, zero2=zero2)
    ex.map_built = True
    for _ in range(2):
        with pytest.raises(RuntimeError):
            ex.clip_gradients(1 << 20, w.ld, 1.0)
        assert not launched and not ex.clip_recs and ex.h_owner is None
    ex.d_owner.copy_(ex.torch.tensor([1, -1, 0]))         # as the replayed build leaves it
    ex.d_pid_off.zero_()
    if zero2:
        ex.d_flat.copy_(ex.torch.tensor([0, 64, 69]))
        ex.d_psize.fill_(51)
    ex.clip_gradients(1 << 20, w.ld, 1.0)
    recs = launched[0]
    at = (recs["grad"].astype(np.int64) - (1 << 20)) // 4
    place = {t.param: bk.col + t.offset for bk in w.buckets for t in bk.tasks}
    got = sorted(zip((at // w.ld).tolist(), (at % w.ld).tolist(), recs["cols"].tolist(), recs["counted"].tolist()))
    if zero2:
        parts = [(0, place[0], 51, 1), (1, place[0] + 51, 13, 1), (1, place[1], 5, 1), (1, place[2], 33, 1)]
    else:
        parts = [(1, place[0], 64, 1), (0, place[1], 5, 1), (1, place[1], 5, 0), (0, place[2], 33, 1)]
    covered = {(r, c + k): counted for r, c, n, counted in got for k in range(n)}
    assert covered == {(r, c + k): counted for r, c, n, counted in parts for k in range(n)}
    assert sum(n for _, _, n, _ in got) == len(covered)


def test_building_again_changes_nothing(launched):
    w, ex = made(reduce_to_owner=True)
    ex.map_built, ex.h_owner = True, np.array([1, -1, 0], np.int32)
    ex.clip_gradients(1 << 20, w.ld, 1.0)
    ex.h_owner = None                                    # as a reader that wants it anew leaves it
    ex.clip_gradients(1 << 20, w.ld, 1.0)
    assert (launched[0] == launched[1]).all()

"""The executor's matrix registration on the host (no GPU): what muon_update
hands to the library, with the launch replaced by a record of it."""
import contextlib

import numpy as np
import pytest
import torch

from gradient_reduction_amd import dc, executor, linear
from synth import workloads as wl

SIZES = [(8, 8), None, (4, 19)]


def made(owners=(1, -1, 0)):
    numel = [a[0] * a[1] if a else 5 for a in SIZES]
    w = wl.custom_flush("update", 2, wl.DT_F32, numel, capacity=9000, pre_div=1, value_seed=3)
    ex = executor.from_workload(w, reduce_to_owner=True, device="cpu")
    ex.h_owner = np.array(owners, np.int32)      # as build_owner_map and fetch_metadata leave it
    place = {t.param: bk.col + t.offset for bk in w.buckets for t in bk.tasks}
    return w, ex, place


def tensors(params=(0, 2)):
    return ({p: torch.zeros(*SIZES[p]) for p in params}, {p: torch.zeros(*SIZES[p]) for p in params})


@pytest.fixture
def launched(monkeypatch):
    """The records of the last dc_muon_update."""
    seen = {}
    monkeypatch.setattr(linear, "on", lambda device, stream: contextlib.nullcontext())
    monkeypatch.setattr(dc, "dc_muon_update", lambda dtype, wtype, held, mats, *rest: seen.update(mats=mats.copy()))
    return seen


def elements(ex, slab, ld, seen):
    ex.muon_update(slab, ld, lr=0.1)
    return ((seen["mats"]["grad"] - slab.data_ptr()) // 4).tolist()


def test_refused_registration_changes_nothing(launched):
    w, ex, place = made()
    slab = torch.zeros(w.W, w.ld)
    ws, ms = tensors()
    ex.register_matrices(ws, ms)
    want = [w.ld + place[0], place[2]]
    assert elements(ex, slab, w.ld, launched) == want
    for bad in [({2: torch.zeros(3, 19)}, {2: torch.zeros(3, 19)}),             # not the param's size
                ({0: torch.zeros(8, 8), 2: torch.zeros(4, 19)}, {0: torch.zeros(8, 8), 2: torch.zeros(4, 18)}),
                ({7: torch.zeros(8, 8)}, {7: torch.zeros(8, 8)}),               # no such param
                ({0: torch.zeros(8, 8)}, {0: torch.zeros(8, 8).double()}),
                ({0: torch.zeros(8, 16)[:, ::2]}, {0: torch.zeros(8, 8)}),
                ({0: torch.zeros(8, 8), 2: torch.zeros(4, 19).bfloat16()}, tensors()[1]),
                ({0: torch.zeros(8, 8)}, {})]:
        with pytest.raises(ValueError):
            ex.register_matrices(*bad)
        assert elements(ex, slab, w.ld, launched) == want
        assert launched["mats"]["out"].tolist() == [ws[0].data_ptr(), ws[2].data_ptr()]
        assert launched["mats"]["momentum"].tolist() == [ms[0].data_ptr(), ms[2].data_ptr()]


def test_a_new_registration_replaces_the_old(launched):
    w, ex, place = made()
    slab = torch.zeros(w.W, w.ld)
    ex.register_matrices(*tensors())
    ex.register_matrices(*tensors([2]))
    assert elements(ex, slab, w.ld, launched) == [place[2]]


def test_registration_needs_the_owner_map(monkeypatch):
    """Before build_owner_map the device map holds nothing: reading it would
    take any row for the owner's."""
    w, ex, place = made()
    ex.h_owner = None
    with pytest.raises(RuntimeError, match="build_owner_map"):
        ex.register_matrices(*tensors())
    assert ex.h_owner is None and ex.m_recs is None
    # with the map built (its launches replaced), it is read back
    monkeypatch.setattr(dc, "dc_partition_ids", lambda *a: None)
    monkeypatch.setattr(dc, "dc_build_owner_map", lambda *a: None)
    ex.build_owner_map()
    ex.d_owner.copy_(torch.tensor([1, -1, 0]))
    ex.d_pid_off.zero_()
    ex.register_matrices(*tensors())
    assert ex.m_rows.tolist() == [1, 0]
    # every row has an AllReduced gradient: no map is needed
    ex = executor.from_workload(w, reduce_to_owner=False, device="cpu")
    ex.register_matrices(*tensors())
    assert ex.m_rows.tolist() == [0, 0]


@pytest.mark.parametrize("as_address", [False, True])
def test_ld_out_is_a_rows_length(launched, as_address):
    """A stride under the row's matrices (or a negative one, which reads before
    the slab) is refused, for a tensor and for an address."""
    w, ex, place = made()
    slab = torch.zeros(w.W, w.ld)
    ex.register_matrices(*tensors())
    least = max(place[0] + 64, place[2] + 76)
    where = slab.data_ptr() if as_address else slab
    for ld in (-w.ld, -1, 0, least - 1):
        with pytest.raises(ValueError, match="ld_out"):
            ex.muon_update(where, ld, lr=0.1)
    assert not launched
    ex.muon_update(where, least, lr=0.1)
    assert ((launched["mats"]["grad"] - slab.data_ptr()) // 4).tolist() == [least + place[0], place[2]]

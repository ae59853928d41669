"""Layers of several replicas into the deferred reduction on streams of their
own: a replica's gradients are in its row whatever the other streams do."""
import pytest
import torch

from gradient_reduction_amd import dc, deferred, executor
from synth import workloads as wl

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    dc.lib()
    yield
    torch.cuda.synchronize()


def test_replicas_on_their_own_streams():
    """Two replicas' layers on two streams, the first one behind other work
    there; small whole numbers, so that every sum is exact."""
    W, t, n, k = 2, 40, 24, 40
    gen = torch.Generator().manual_seed(2)
    red = deferred.DeferredReducer(W, n * k + 100)
    streams = [torch.cuda.Stream() for _ in range(W)]
    busy = torch.ones(4096, 4096, device="cuda")
    w = torch.ones(n, k, device="cuda")
    for step in range(3):
        red.acc.fill_(7.0)
        x = torch.randint(-3, 4, (W, 2, t, k), generator=gen).float().cuda()
        dy = torch.randint(-3, 4, (W, 2, t, n), generator=gen).float().cuda()
        torch.cuda.synchronize()
        for mb in range(2):
            for r in range(W):
                if r == 0:
                    with torch.cuda.stream(streams[0]):
                        for _ in range(3):
                            busy = busy @ busy * 2.0 ** -12
                red.accumulate_linear(r, 5, dy[r, mb], x[r, mb], w, stream=streams[r])
            red.end_micro_batch()
        for s in streams:
            torch.cuda.current_stream().wait_stream(s)
        out = torch.zeros(1, red.ld, device="cuda")
        red.reduce(out, red.ld)
        for r in range(W):
            want = sum(dy[r, mb].double().t() @ x[r, mb].double() for mb in range(2))
            assert torch.equal(red.acc[r, 5:5 + n * k].view(n, k).double(), want), (step, r)
            assert not red.acc[r, :5].any() and not red.acc[r, 5 + n * k:].any()
        total = red.acc.double().sum(0)
        assert torch.equal(out[0, :red.M].double(), total[:red.M])


def test_a_replica_without_layers():
    red = deferred.DeferredReducer(3, 24 * 40)
    red.acc.fill_(float("nan"))
    x, dy, w = torch.ones(2, 40, device="cuda"), torch.ones(2, 24, device="cuda"), torch.ones(24, 40, device="cuda")
    red.accumulate_linear(1, 0, dy, x, w)
    red.end_micro_batch()
    red.accumulate_linear(0, 0, dy, x, w)
    red.end_micro_batch()
    out = torch.zeros(3, red.ld, device="cuda")
    red.reduce(out, red.ld, out_rows=3)
    acc = red.acc.cpu()
    assert bool((acc[0] == 2).all()) and bool((acc[1] == 2).all()) and not acc[2].any()
    assert bool(torch.isfinite(out).all()) and torch.equal(out[0], out[2])


def test_registration_waits_for_an_owner_map_on_another_stream():
    """The map is built behind other work on a side stream; the matrices'
    rows are the owners that it gives."""
    sizes = [(40, 30), (64, 64), (7, 200), (90, 11)]
    w = wl.custom_flush("update", 4, wl.DT_F32, [a * b for a, b in sizes], capacity=9000, pre_div=1, value_seed=3)
    plain = executor.from_workload(w, reduce_to_owner=True)
    plain.build_owner_map()
    plain.fetch_metadata()
    ex = executor.from_workload(w, reduce_to_owner=True)
    ex.d_owner.fill_(-1)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    busy = torch.ones(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(20):
            busy = busy @ busy * 2.0 ** -12
    ex.build_owner_map(stream=side.cuda_stream)
    ts = {p: torch.zeros(*s, device="cuda") for p, s in enumerate(sizes)}
    ex.register_matrices(ts, {p: torch.zeros_like(v) for p, v in ts.items()})
    assert plain.h_owner.max() > 0 and ex.h_owner.tolist() == plain.h_owner.tolist()
    assert ex.m_rows.tolist() == [max(int(o), 0) for o in plain.h_owner]

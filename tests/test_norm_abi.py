"""The norms' entry points on the host (no GPU): refusals and workspaces."""
import contextlib

import pytest
import torch

from gradient_reduction_amd import dc, deferred, linear, norm
from tests.test_abi import FAKE, expect

FAR = 1 << 36


def at(k):
    return FAKE + k * FAR


FORWARD = dict(dtype=0, T=6, D=5, x=at(0), ld_x=5, h=at(1), ld_h=5, post_gain=at(2), gate=at(3), gate_rows=2, ld_gate=5,
               gain=at(4), scale=1.0, offset=0.0, eps=1e-6, s=at(5), ld_s=5, y=at(6), ld_y=5, stream=0)
COMMON = [
    (dc.DC_ERR_DTYPE, dict(dtype=2)), (dc.DC_ERR_ARG, dict(T=-2)), (dc.DC_ERR_ARG, dict(D=0)),
    (dc.DC_ERR_UNSUPPORTED, dict(D=16385)), (dc.DC_ERR_SHAPE, dict(T=(1 << 28) + 2)),
    (dc.DC_ERR_ARG, dict(gate_rows=0)), (dc.DC_ERR_SHAPE, dict(gate_rows=4)), (dc.DC_ERR_ARG, dict(scale=float("nan"))),
    (dc.DC_ERR_ARG, dict(offset=float("inf"))), (dc.DC_ERR_ARG, dict(eps=-1e-6)), (dc.DC_ERR_ARG, dict(eps=float("nan"))),
    (dc.DC_ERR_NULL, dict(h=None)), (dc.DC_ERR_ALIGN, dict(h=at(1) + 1)), (dc.DC_ERR_ALIGN, dict(gain=at(4) + 1)),
    (dc.DC_ERR_SHAPE, dict(ld_h=4)), (dc.DC_ERR_SHAPE, dict(ld_gate=4)), (dc.DC_ERR_ALIGN, dict(post_gain=at(2) + 1)),
]


@pytest.mark.parametrize("code, change", COMMON + [
    (dc.DC_ERR_NULL, dict(x=None)), (dc.DC_ERR_NULL, dict(y=None)), (dc.DC_ERR_NULL, dict(gain=None)),
    (dc.DC_ERR_NULL, dict(s=None, y=None, gain=None)), (dc.DC_ERR_NULL, dict(h=None, post_gain=None, gate=None)),
    (dc.DC_ERR_SHAPE, dict(ld_x=4)), (dc.DC_ERR_SHAPE, dict(ld_s=4)), (dc.DC_ERR_SHAPE, dict(ld_y=4)),
    (dc.DC_ERR_ARG, dict(s=at(0) + 2)), (dc.DC_ERR_ARG, dict(s=at(0), ld_s=6)), (dc.DC_ERR_ARG, dict(y=at(5))),
    (dc.DC_ERR_ARG, dict(s=at(2))), (dc.DC_ERR_ARG, dict(y=at(4) + 2)), (dc.DC_ERR_ARG, dict(y=at(1), ld_y=7)),
    (dc.DC_ERR_ARG, dict(s=at(3))),
])
def test_forward_refusals(code, change):
    expect(code, dc.dc_norm, **{**FORWARD, **change})


BACK = dict(dtype=0, T=6, D=5, dy=at(0), ld_dy=5, ds=at(1), ld_ds=5, s=at(2), ld_s=5, h=at(3), ld_h=5, post_gain=at(4),
            gate=at(5), gate_rows=2, ld_gate=5, gain=at(6), scale=1.0, offset=0.0, eps=1e-6, dx=at(7), ld_dx=5, dh=at(8),
            ld_dh=5, grad_dtype=1, dgain=at(9), dpost_gain=at(10), dgate=at(11), ld_dgate=5, accumulate=1,
            workspace=at(12), workspace_bytes=1 << 30, stream=0)


@pytest.mark.parametrize("code, change", [c for c in COMMON if c[1] != dict(h=at(1) + 1)] + [
    (dc.DC_ERR_ALIGN, dict(h=at(3) + 1)), (dc.DC_ERR_DTYPE, dict(grad_dtype=2)),
    (dc.DC_ERR_DTYPE, dict(dtype=1, grad_dtype=0)), (dc.DC_ERR_ARG, dict(accumulate=2)),
    (dc.DC_ERR_NULL, dict(dy=None)), (dc.DC_ERR_NULL, dict(s=None)), (dc.DC_ERR_NULL, dict(gain=None)),
    (dc.DC_ERR_NULL, dict(post_gain=None)), (dc.DC_ERR_NULL, dict(gate=None)),
    (dc.DC_ERR_NULL, dict(dx=None, dh=None, dgain=None, dpost_gain=None, dgate=None)),
    (dc.DC_ERR_NULL, dict(h=None, post_gain=None, gate=None)),
    (dc.DC_ERR_NULL, dict(h=None, post_gain=None, gate=None, gain=None, dh=None, dgain=None, dpost_gain=None, dgate=None)),
    (dc.DC_ERR_SHAPE, dict(ld_dx=4)), (dc.DC_ERR_SHAPE, dict(ld_dh=4)), (dc.DC_ERR_SHAPE, dict(ld_dgate=4)),
    (dc.DC_ERR_SHAPE, dict(ld_dy=4)), (dc.DC_ERR_SHAPE, dict(ld_ds=4)), (dc.DC_ERR_SHAPE, dict(ld_s=4)),
    (dc.DC_ERR_ALIGN, dict(dgain=at(9) + 2)), (dc.DC_ERR_ARG, dict(dx=at(0) + 2)), (dc.DC_ERR_ARG, dict(dx=at(1), ld_dx=6)),
    (dc.DC_ERR_ARG, dict(dh=at(7))), (dc.DC_ERR_ARG, dict(dx=at(6))), (dc.DC_ERR_ARG, dict(dgain=at(0))),
    (dc.DC_ERR_ARG, dict(dpost_gain=at(9) + 4)), (dc.DC_ERR_ARG, dict(dgate=at(10) - 4)), (dc.DC_ERR_ARG, dict(dgate=at(3))),
    (dc.DC_ERR_SHAPE, dict(workspace_bytes=8)), (dc.DC_ERR_NULL, dict(workspace=None)),
    (dc.DC_ERR_ALIGN, dict(workspace=at(12) + 4)),
])
def test_backward_refusals(code, change):
    expect(code, dc.dc_norm_backward, **{**BACK, **change})


def test_workspaces():
    need = dc.dc_norm_backward_workspace
    assert need(0, 0, 5, 1) >= 0 and need(0, 8192, 4096, 1) >= 2 * 4 * 4096
    assert need(0, 8192, 4096, 8192) > need(0, 8192, 4096, 1) and need(0, 4, 64, 1) <= 1 << 20
    assert all(need(k, t, d, 1) < 1 << 27 for k in (0, 1) for t in (1, 1000, 1 << 20) for d in (1, 1000, 16384))
    expect(dc.DC_ERR_NULL, lambda: dc._check("q", dc.lib().dc_norm_backward_workspace(0, 1, 1, 1, None)))
    for bad in ((2, 1, 1, 1), (0, -1, 1, 1), (0, 1, 0, 1), (0, 1, 1, 0), (0, 3, 1, 2), (0, 1, 16385, 1)):
        with pytest.raises(dc.DCError):
            need(*bad)


def test_python_refusals():
    x, w = torch.zeros(6, 5), torch.zeros(5)
    for a, kw in [((x, w), {}), ((x,), {}), ((x.half(), w.half()), {}), ((x, w[:4]), {}), ((x, w.bfloat16()), {}),
                  ((x, w), dict(post_gain=w)), ((x, w), dict(gate=w)), ((x, w), dict(h=x[:3])), ((x.t(), w), {}),
                  ((x, w), dict(h=x, gate=torch.zeros(4, 5))), ((x, w), dict(h=x, gate=torch.zeros(2, 3, 5))),
                  ((x, w), dict(h=x, gate=torch.zeros(0, 5))), ((x, w), dict(eps=-1.0)), ((x, w), dict(eps=float("nan"))),
                  ((x, w), dict(offset=float("inf"))), ((x, w), dict(out=x)), ((x,), dict(h=x, out_norm=x)),
                  ((torch.zeros(()), w), {}), ((torch.zeros(2, 3, 5)[:, 1:], w), {})]:
        with pytest.raises(ValueError):
            norm.forward(*a, **kw)


@pytest.fixture
def launches(monkeypatch):
    seen = []
    monkeypatch.setattr(norm, "on", lambda device, stream: contextlib.nullcontext())
    monkeypatch.setattr(linear, "on", lambda device, stream: contextlib.nullcontext())
    monkeypatch.setattr(dc, "dc_norm_backward", lambda *a: seen.append(a))
    return seen


def test_backward_refuses_before_anything_is_launched(launches):
    x, w, g = torch.zeros(6, 5), torch.zeros(5), torch.zeros(2, 5)
    ok = dict(dy=x, s=x, gain=w, ds=x, h=x, post_gain=w, gate=g)
    wide = torch.zeros(6, 12)
    for kw in (dict(dy=None), dict(dy=x[:3]), dict(ds=x.bfloat16()), dict(gain=None, dgain=w.clone()),
               dict(accumulate=True), dict(dgain=w), dict(dgain=torch.zeros(5).double()), dict(dgate=torch.zeros(5)),
               dict(dgate=torch.zeros(2, 5), dgain=torch.zeros(5), dpost_gain=torch.zeros(5).bfloat16()),
               dict(dgain=wide.view(-1)[:5], dpost_gain=wide.view(-1)[4:9]), dict(dgate=x[:2]),
               dict(dgate=torch.zeros(4, 5)[::2].t().contiguous().t()), dict(scale=float("nan"))):
        with pytest.raises(ValueError):
            norm.backward(**{**ok, **kw})
        assert not launches
    norm.backward(**ok)
    norm.backward(**ok, dgate=wide[:2, 3:8], dgain=wide[5, :5], dpost_gain=wide[4, :5], accumulate=True)
    assert len(launches) == 2
    norm.backward(**{**ok, "gain": None, "dy": None}, need_params=False, need_dx=False, need_dh=False)
    assert len(launches) == 2                                 # nothing is wanted


def test_a_refused_layer_leaves_the_accumulators(launches):
    d = deferred.DeferredReducer(2, 100, device="cpu")
    d.acc.fill_(7.0)
    x, w, g = torch.zeros(6, 5), torch.zeros(5), torch.zeros(2, 5)
    ok = dict(row=0, dy=x, s=x, gain=w, h=x, post_gain=w, gate=g, gain_at=0, post_gain_at=5, gate_at=10)
    over = torch.as_strided(d.acc, (6, 5), (5, 1), 12)
    for kw in (dict(row=2), dict(row=-1), dict(gain_at=96), dict(post_gain_at=4), dict(gate_at=9), dict(dy=over),
               dict(h=None), dict(gate=None), dict(eps=-1.0), dict(dy=x.double())):
        with pytest.raises(ValueError):
            d.accumulate_norm(**{**ok, **kw})
        assert not launches and bool((d.acc == 7).all()) and not d.open
    d.accumulate_norm(**ok)
    assert len(launches) == 1 and d.open and not d.acc[0].any() and bool((d.acc[1] == 7).all())

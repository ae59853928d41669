"""Clipping's entry points on the host (no GPU): every argument check returns
its documented code before any device work, the records that the Python layer
makes, and its refusals."""
import numpy as np
import pytest
import torch

from gradient_reduction_amd import clip, dc, deferred
from tests.test_abi import FAKE, expect

FAR = 1 << 34


def at(k):
    return FAKE + k * FAR


def grads(*specs, **change):
    r = np.zeros(len(specs), dc.GRADIENT_DTYPE)
    for k, (rows, cols) in enumerate(specs):
        r[k] = (at(2 * k), at(2 * k + 1), cols, cols, rows, cols, rows, 0, 0)
    for name, (k, v) in change.items():
        r[name][k] = v
    return r


def call(m=grads((3, 4)), num=None, squares=at(20), max_norm=1.0, eps=1e-6, norm=at(21), coef=at(22), ws=at(23),
         nbytes=1 << 20):
    dc.dc_grad_clip(m, len(m) if num is None and m is not None else num, squares, max_norm, eps, norm, coef, ws,
                    nbytes, 0)


def norm_call(m=grads((3, 4)), num=None, accumulate=0, squares=at(20), norm=at(21), ws=at(23), nbytes=1 << 20):
    dc.dc_grad_norm(m, len(m) if num is None and m is not None else num, accumulate, squares, norm, ws, nbytes, 0)


BOTH = [
    (dc.DC_ERR_ARG, dict(num=-1)), (dc.DC_ERR_ARG, dict(num=(1 << 20) + 1)), (dc.DC_ERR_NULL, dict(m=None, num=1)),
    (dc.DC_ERR_DTYPE, dict(m=grads((3, 4), dtype=(0, 2)))), (dc.DC_ERR_ARG, dict(m=grads((-1, 4)))),
    (dc.DC_ERR_ARG, dict(m=grads((3, -4)))), (dc.DC_ERR_ARG, dict(m=grads((3, 4), counted=(0, 4)))),
    (dc.DC_ERR_ARG, dict(m=grads((3, 4), counted=(0, -1)))), (dc.DC_ERR_SHAPE, dict(m=grads(((1 << 36) + 1, 1)))),
    (dc.DC_ERR_SHAPE, dict(m=grads((1, (1 << 36) + 1)))), (dc.DC_ERR_SHAPE, dict(m=grads((1 << 20, 1 << 17)))),
    (dc.DC_ERR_NULL, dict(m=grads((3, 4), grad=(0, 0)))), (dc.DC_ERR_SHAPE, dict(m=grads((3, 4), ld_grad=(0, 3)))),
    (dc.DC_ERR_SHAPE, dict(m=grads((3, 4), ld_grad=(0, 1 << 45)))),
    (dc.DC_ERR_ALIGN, dict(m=grads((3, 4), grad=(0, at(0) + 1)))), (dc.DC_ERR_ALIGN, dict(squares=at(20) + 4)),
    (dc.DC_ERR_ALIGN, dict(norm=at(21) + 2)), (dc.DC_ERR_ARG, dict(norm=at(0) + 4)),
    (dc.DC_ERR_ARG, dict(norm=at(20) + 4)), (dc.DC_ERR_SHAPE, dict(nbytes=100)), (dc.DC_ERR_NULL, dict(ws=None)),
    (dc.DC_ERR_ALIGN, dict(ws=at(23) + 8)),
]


@pytest.mark.parametrize("code, change", BOTH + [
    (dc.DC_ERR_ARG, dict(max_norm=-1.0)), (dc.DC_ERR_ARG, dict(max_norm=float("nan"))),
    (dc.DC_ERR_ARG, dict(eps=-1.0)), (dc.DC_ERR_ARG, dict(eps=float("inf"))),
    (dc.DC_ERR_ALIGN, dict(coef=at(22) + 1)), (dc.DC_ERR_ARG, dict(coef=at(21))),
    (dc.DC_ERR_ARG, dict(squares=at(1))), (dc.DC_ERR_ARG, dict(coef=at(1) + 4)),
    (dc.DC_ERR_NULL, dict(m=grads((3, 4), out=(0, 0)))), (dc.DC_ERR_SHAPE, dict(m=grads((3, 4), ld_out=(0, 3)))),
    (dc.DC_ERR_ARG, dict(m=grads((3, 4), (3, 4), out=(1, at(1))))),           # one output twice
    (dc.DC_ERR_ARG, dict(m=grads((3, 4), (3, 4), out=(1, at(1) + 20)))),      # shared tail
    (dc.DC_ERR_ARG, dict(m=grads((3, 4), (3, 4), out=(1, at(0))))),           # another one's gradient
    (dc.DC_ERR_ARG, dict(m=grads((3, 4), out=(0, at(0) + 2)))),               # its own, shifted
    (dc.DC_ERR_ARG, dict(m=grads((3, 4), out=(0, at(0)), ld_out=(0, 5)))),    # its own, another stride
])
def test_clip_refusals(code, change):
    expect(code, call, **change)


@pytest.mark.parametrize("code, change", BOTH + [
    (dc.DC_ERR_ARG, dict(accumulate=2)), (dc.DC_ERR_NULL, dict(squares=None, norm=None)),
    (dc.DC_ERR_NULL, dict(squares=None, accumulate=1)), (dc.DC_ERR_ARG, dict(squares=at(0))),
])
def test_norm_refusals(code, change):
    expect(code, norm_call, **change)


def test_one_gradient_twice():
    """In place the second scaling would meet the first: refused.  The norm
    alone may count one twice (the check passes on to the workspace's)."""
    two = grads((3, 4), (3, 4), grad=(1, at(0)))
    two["out"] = two["grad"]
    expect(dc.DC_ERR_ARG, call, m=two)
    expect(dc.DC_ERR_SHAPE, norm_call, m=two, nbytes=0)


def test_workspace_and_layout():
    assert dc.GRADIENT_DTYPE.itemsize == 64
    assert 0 < dc.dc_grad_clip_workspace() <= 1 << 20
    expect(dc.DC_ERR_NULL, lambda: dc._check("q", dc.lib().dc_grad_clip_workspace(None)))


def test_records():
    def runs(t):
        return clip._runs("t", t)

    a = torch.zeros(4, 5, 6)
    assert runs(a) == (1, 120, 120) and runs(a.permute(2, 0, 1)) == (1, 120, 120)
    assert runs(a[:, :, :3]) == (20, 3, 6) and runs(a[:, :2]) == (4, 12, 30) and runs(a[::2]) == (2, 30, 60)
    assert runs(a[1, 2, 3]) == (1, 1, 1) and runs(torch.zeros(())) == (1, 1, 1) and runs(a[:0]) == (0, 0, 0)
    assert runs(torch.zeros(7, 3)[:, 1]) == (7, 1, 3)
    for bad in (a[:, ::2, ::2], a[:1].expand(3, 5, 6), torch.zeros(8).as_strided((3, 4), (2, 1))):
        with pytest.raises(ValueError):
            runs(bad)
    r = clip.gradients([a[:, :2], torch.zeros(3).bfloat16()], [torch.zeros(4, 2, 6), torch.zeros(3).bfloat16()])
    assert r["rows"].tolist() == [4, 1] and r["cols"].tolist() == [12, 3] and r["ld_grad"].tolist() == [30, 3]
    assert r["ld_out"].tolist() == [12, 3] and r["dtype"].tolist() == [1, 0] and r["counted"].tolist() == [4, 1]
    r = clip.gradients([torch.zeros(4, 2, 6)], [a[:, :2]])
    assert (r["rows"][0], r["cols"][0], r["ld_grad"][0], r["ld_out"][0]) == (4, 12, 12, 30)


def test_python_refusals():
    a = torch.zeros(4, 6)
    for args in (([],), ([a],), ([a.half()],), ([a[::2, ::2]],)):
        with pytest.raises(ValueError):
            clip.grad_norm(*args)
        with pytest.raises(ValueError):
            clip.clip_grad_norm(*args, 1.0)
    for kw in (dict(out=[]), dict(out=[a.bfloat16()]), dict(out=[torch.zeros(4, 5)]), dict(out=[torch.zeros(6, 4).t()]),
               dict(squares=torch.zeros(1)), dict(squares=torch.zeros(2).double())):
        with pytest.raises(ValueError):
            clip.clip_grad_norm([a], 1.0, **kw)
    with pytest.raises(ValueError):
        clip.sum_squares([a], accumulate=True)
    d = deferred.DeferredReducer(2, 40, device="cpu")
    for kw in (dict(ld_out=39), dict(out_rows=3), dict(out=torch.zeros(30)), dict(out=torch.zeros(64).double())):
        with pytest.raises(ValueError):
            d.clip(**{**dict(out=torch.zeros(64), ld_out=64, max_norm=1.0), **kw})

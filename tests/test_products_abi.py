"""The linear layer's, the orthogonalisation's and the update's entry points on
the host (no GPU): every argument check returns its documented code before any
device work, workspace queries, and the Python layer's refusals."""
import numpy as np
import pytest
import torch

from gradient_reduction_amd import dc, deferred, linear, muon
from tests.test_abi import FAKE, expect

COEFFS = np.tile(np.array(muon.COEFFS, np.float32), (5, 1))
FAR = 1 << 34     # between fake operands that must not overlap


def at(k):
    return FAKE + k * FAR


LINEAR = dict(dtype=0, T=4, N=6, K=5, x=at(0), ld_x=5, w=at(1), ld_w=5, bias=at(2), residual=at(3), ld_res=6,
              act=2, pre=at(4), ld_pre=6, y=at(5), ld_y=6, workspace=at(6), workspace_bytes=1 << 30, stream=0)


@pytest.mark.parametrize("code, change", [
    (dc.DC_ERR_DTYPE, dict(dtype=2)), (dc.DC_ERR_ARG, dict(T=-1)), (dc.DC_ERR_ARG, dict(N=0)),
    (dc.DC_ERR_ARG, dict(K=0)), (dc.DC_ERR_SHAPE, dict(T=(1 << 28) + 1)),
    (dc.DC_ERR_SHAPE, dict(T=1 << 20, N=1 << 20, ld_y=1 << 20, ld_pre=1 << 20, ld_res=1 << 20)),
    (dc.DC_ERR_ARG, dict(act=4)), (dc.DC_ERR_ARG, dict(act=-1)),
    (dc.DC_ERR_NULL, dict(x=None)), (dc.DC_ERR_NULL, dict(w=None)), (dc.DC_ERR_NULL, dict(y=None)),
    (dc.DC_ERR_SHAPE, dict(ld_x=4)), (dc.DC_ERR_SHAPE, dict(ld_w=4)), (dc.DC_ERR_SHAPE, dict(ld_y=5)),
    (dc.DC_ERR_SHAPE, dict(ld_pre=5)), (dc.DC_ERR_SHAPE, dict(ld_res=5)), (dc.DC_ERR_SHAPE, dict(ld_x=1 << 45)),
    (dc.DC_ERR_ALIGN, dict(x=at(0) + 1)), (dc.DC_ERR_ALIGN, dict(bias=at(2) + 1)),
    (dc.DC_ERR_ARG, dict(y=at(0) + 2)), (dc.DC_ERR_ARG, dict(y=at(1))), (dc.DC_ERR_ARG, dict(pre=at(5) + 4)),
    (dc.DC_ERR_ARG, dict(residual=at(5) + 2)), (dc.DC_ERR_ARG, dict(residual=at(5), ld_res=7)),
    (dc.DC_ERR_ARG, dict(pre=at(3))), (dc.DC_ERR_ARG, dict(y=at(2) + 2)),
])
def test_linear_refusals(code, change):
    expect(code, dc.dc_linear, **{**LINEAR, **change})


BIAS = dict(dtype=0, T=4, N=6, dy=at(0), ld_dy=6, pre=at(1), ld_pre=6, act=2, dz=at(2), ld_dz=6, grad_dtype=1,
            db=at(3), accumulate=0, workspace=at(4), workspace_bytes=1 << 30, stream=0)


@pytest.mark.parametrize("code, change", [
    (dc.DC_ERR_DTYPE, dict(dtype=7)), (dc.DC_ERR_DTYPE, dict(grad_dtype=2)),
    (dc.DC_ERR_DTYPE, dict(dtype=1, grad_dtype=0)), (dc.DC_ERR_ARG, dict(accumulate=2)),
    (dc.DC_ERR_NULL, dict(dz=None, db=None)), (dc.DC_ERR_NULL, dict(dy=None)), (dc.DC_ERR_NULL, dict(pre=None)),
    (dc.DC_ERR_SHAPE, dict(ld_pre=5)), (dc.DC_ERR_SHAPE, dict(ld_dz=5)), (dc.DC_ERR_ALIGN, dict(db=at(3) + 2)),
    (dc.DC_ERR_ARG, dict(dz=at(0) + 2)), (dc.DC_ERR_ARG, dict(dz=at(0), ld_dz=8)), (dc.DC_ERR_ARG, dict(dz=at(1))),
    (dc.DC_ERR_ARG, dict(db=at(0))), (dc.DC_ERR_ARG, dict(db=at(2))), (dc.DC_ERR_ARG, dict(T=-1)),
    (dc.DC_ERR_ARG, dict(N=0)), (dc.DC_ERR_ARG, dict(act=9)),
])
def test_bias_act_refusals(code, change):
    expect(code, dc.dc_bias_act_backward, **{**BIAS, **change})


BACK = dict(dtype=0, T=4, N=6, K=5, dz=at(0), ld_dz=6, w=at(1), ld_w=5, x=at(2), ld_x=5, dx=at(3), ld_dx=5,
            grad_dtype=1, dw=at(4), ld_dw=5, accumulate=1, workspace=at(5), workspace_bytes=1 << 30, stream=0)


@pytest.mark.parametrize("code, change", [
    (dc.DC_ERR_DTYPE, dict(dtype=3)), (dc.DC_ERR_DTYPE, dict(dtype=1, grad_dtype=0)),
    (dc.DC_ERR_NULL, dict(dx=None, dw=None)), (dc.DC_ERR_NULL, dict(dz=None)), (dc.DC_ERR_NULL, dict(w=None)),
    (dc.DC_ERR_NULL, dict(x=None)), (dc.DC_ERR_ARG, dict(accumulate=-1)), (dc.DC_ERR_SHAPE, dict(ld_dw=4)),
    (dc.DC_ERR_SHAPE, dict(ld_dx=4)), (dc.DC_ERR_SHAPE, dict(ld_dz=5)), (dc.DC_ERR_ALIGN, dict(dw=at(4) + 2)),
    (dc.DC_ERR_ARG, dict(dx=at(0))), (dc.DC_ERR_ARG, dict(dw=at(3))), (dc.DC_ERR_ARG, dict(dx=at(2))),
    (dc.DC_ERR_ARG, dict(dw=at(1), grad_dtype=0)),
])
def test_linear_backward_refusals(code, change):
    expect(code, dc.dc_linear_backward, **{**BACK, **change})


def mats(*specs, **change):
    r = np.zeros(len(specs), dc.MATRIX_DTYPE)
    for k, (rows, cols) in enumerate(specs):
        r[k] = (at(3 * k), at(3 * k + 1), at(3 * k + 2), cols, cols, rows, cols)
    for name, (k, v) in change.items():
        r[name][k] = v
    return r


BIG = 1 << 40


@pytest.mark.parametrize("code, m", [
    (dc.DC_ERR_ARG, mats((0, 3))), (dc.DC_ERR_ARG, mats((3, -1))), (dc.DC_ERR_SHAPE, mats((1 << 18, 1 << 17))),
    (dc.DC_ERR_SHAPE, mats(((1 << 28) + 1, 1))), (dc.DC_ERR_NULL, mats((3, 4), grad=(0, 0))),
    (dc.DC_ERR_NULL, mats((3, 4), out=(0, 0))), (dc.DC_ERR_SHAPE, mats((3, 4), ld_grad=(0, 3))),
    (dc.DC_ERR_SHAPE, mats((3, 4), ld_out=(0, 3))), (dc.DC_ERR_ALIGN, mats((3, 4), grad=(0, at(0) + 1))),
    (dc.DC_ERR_ARG, mats((3, 4), (3, 4), out=(1, at(1)))),           # one output twice
    (dc.DC_ERR_ARG, mats((3, 4), (3, 4), out=(1, at(1) + 20))),      # shared tail
    (dc.DC_ERR_ARG, mats((3, 4), (3, 4), out=(1, at(0)))),           # another matrix's gradient
    (dc.DC_ERR_ARG, mats((3, 4), out=(0, at(0) + 2))),               # its own, shifted
])
def test_list_refusals(code, m):
    expect(code, dc.dc_orthogonalize, 0, 0, m, len(m), 5, COEFFS, 1e-7, at(20), BIG, 0)
    if not (len(m) == 1 and m["out"][0] == m["grad"][0] + 2):
        expect(code, dc.dc_muon_update, 0, 0, 0, m, len(m), 0.1, None, 0.9, 1, 0.0, 2, 5, COEFFS, 1e-7, at(20), BIG, 0)


def test_update_refusals():
    def call(m=mats((3, 4)), dtype=0, wtype=1, hold=0, num=1, lr=0.1, lrs=None, mu=0.9, nest=1, wd=0.0, mode=2, steps=5,
             co=COEFFS, eps=1e-7, ws=at(20), nbytes=BIG):
        dc.dc_muon_update(dtype, wtype, hold, m, num, lr, lrs, mu, nest, wd, mode, steps, co, eps, ws, nbytes, 0)

    for code, change in [(dc.DC_ERR_DTYPE, dict(dtype=2)), (dc.DC_ERR_DTYPE, dict(wtype=-1)),
                         (dc.DC_ERR_ARG, dict(hold=3)), (dc.DC_ERR_ARG, dict(hold=-1)),
                         (dc.DC_ERR_ARG, dict(lr=float("nan"))), (dc.DC_ERR_ARG, dict(mu=float("inf"))),
                         (dc.DC_ERR_ARG, dict(wd=float("nan"))), (dc.DC_ERR_ARG, dict(nest=2)),
                         (dc.DC_ERR_ARG, dict(mode=3)), (dc.DC_ERR_ARG, dict(steps=0)),
                         (dc.DC_ERR_ARG, dict(steps=17)), (dc.DC_ERR_NULL, dict(co=None)),
                         (dc.DC_ERR_ARG, dict(eps=-1.0)), (dc.DC_ERR_ARG, dict(eps=float("nan"))),
                         (dc.DC_ERR_ARG, dict(num=-1)), (dc.DC_ERR_NULL, dict(m=None)),
                         (dc.DC_ERR_ALIGN, dict(lrs=at(21) + 2)), (dc.DC_ERR_SHAPE, dict(nbytes=100)),
                         (dc.DC_ERR_NULL, dict(ws=None)), (dc.DC_ERR_ALIGN, dict(ws=at(20) + 8)),
                         (dc.DC_ERR_NULL, dict(m=mats((3, 4), momentum=(0, 0)))),
                         (dc.DC_ERR_ARG, dict(m=mats((3, 4), momentum=(0, at(0))))),
                         (dc.DC_ERR_ARG, dict(m=mats((3, 4), momentum=(0, at(1))))),
                         (dc.DC_ERR_ARG, dict(m=mats((3, 4), out=(0, at(0))), wtype=0))]:
        expect(code, call, **change)


@pytest.mark.parametrize("co", [
    np.tile(np.array([10.0, 0.0, 0.0], np.float32), (5, 1)),     # 10^5
    np.tile(np.array([1.0, 5.0, 0.0], np.float32), (5, 1)),
    np.array([[np.nan, 0, 0]], np.float32), np.array([[1, np.inf, 0]], np.float32),
])
def test_diverging_steps_are_refused(co):
    m = mats((3, 4))
    expect(dc.DC_ERR_ARG, dc.dc_orthogonalize, 0, 0, m, 1, len(co), co, 1e-7, at(20), BIG, 0)


def test_interleaved_columns_do_not_overlap():
    """Column ranges of rows with one stride: the check passes them on to the
    workspace's (which is too small here), and refuses one column more."""
    m = mats((8, 4), (8, 4))
    m["ld_out"] = 8
    m["out"] = at(1), at(1) + 8
    expect(dc.DC_ERR_SHAPE, dc.dc_orthogonalize, 0, 0, m, 2, 5, COEFFS, 1e-7, at(20), 16, 0)
    m["out"][1] = at(1) + 6
    expect(dc.DC_ERR_ARG, dc.dc_orthogonalize, 0, 0, m, 2, 5, COEFFS, 1e-7, at(20), 16, 0)
    m["out"][1] = at(1) + 10      # wraps into the next row's first column
    expect(dc.DC_ERR_ARG, dc.dc_orthogonalize, 0, 0, m, 2, 5, COEFFS, 1e-7, at(20), 16, 0)


def test_workspaces():
    assert dc.dc_orthogonalize_workspace(0, 0, 0, mats(), 0) == 0
    one = dc.dc_orthogonalize_workspace(0, 0, 0, mats((400, 300)), 1)
    assert one >= 2 * (2 * 400 * 300 + 2 * 300 * 300)
    pair = dc.dc_orthogonalize_workspace(1, 1, 0, mats((400, 300)), 1)
    assert pair > one and pair == dc.dc_orthogonalize_workspace(0, 1, 0, mats((400, 300)), 1)
    assert pair == dc.dc_orthogonalize_workspace(0, 0, 2, mats((400, 300)), 1)
    assert one == dc.dc_orthogonalize_workspace(1, 1, 1, mats((400, 300)), 1)
    for bad in ((2, 0, 0), (0, 2, 0), (0, 0, 3)):
        with pytest.raises(dc.DCError):
            dc.dc_orthogonalize_workspace(*bad, mats((400, 300)), 1)
    many = np.concatenate([mats((400, 300))] * 1000)     # chunks reuse the workspace
    assert dc.dc_orthogonalize_workspace(0, 0, 0, many, 1000) < 200 * one
    assert dc.dc_linear_workspace(0, 8192, 8192, 64) == 0
    for T, N, K in [(1, 1, 1), (64, 64, 100000), (7, 300, 5000)]:
        assert dc.dc_linear_workspace(1, T, N, K) % 16 == 0
        need = dc.dc_linear_workspace(0, T, N, K)
        if need:
            big = {**LINEAR, "T": T, "N": N, "K": K, "ld_x": K, "ld_w": K, "ld_res": N, "ld_pre": N, "ld_y": N}
            expect(dc.DC_ERR_SHAPE, dc.dc_linear, **{**big, "workspace_bytes": need - 1})
            expect(dc.DC_ERR_NULL, dc.dc_linear, **{**big, "workspace": None})
            expect(dc.DC_ERR_ALIGN, dc.dc_linear, **{**big, "workspace": at(6) + 4})
    expect(dc.DC_ERR_NULL, lambda: dc._check("q", dc.lib().dc_linear_workspace(0, 1, 1, 1, None)))
    assert dc.dc_bias_act_workspace(0, 0, 5) == 0 and dc.dc_linear_backward_workspace(0, 0, 5, 5) == 0


def test_matrix_record_layout():
    assert dc.MATRIX_DTYPE.itemsize == 48


def test_python_refusals():
    x, w = torch.zeros(4, 5), torch.zeros(6, 5)
    with pytest.raises(ValueError):
        linear.forward(x, w)                                   # no GPU tensors
    with pytest.raises(ValueError):
        linear.forward(x, w, act="tanh")
    with pytest.raises(ValueError):
        linear.forward(x, torch.zeros(6, 4))
    with pytest.raises(ValueError):
        linear.forward(x.half(), w.half())
    with pytest.raises(ValueError):
        linear.forward(x.t(), torch.zeros(6, 4))               # strided columns
    with pytest.raises(ValueError):
        linear.forward(torch.zeros(1, 5).expand(4, 5), w)      # broadcast rows
    with pytest.raises(ValueError):
        linear.bias_act_backward(torch.zeros(4, 6), act="gelu")
    with pytest.raises(ValueError):
        linear.backward(torch.zeros(4, 6), x, w, accumulate=True)
    g = torch.zeros(3, 4)
    with pytest.raises(ValueError):
        muon.orthogonalize(g)
    with pytest.raises(ValueError):
        muon.orthogonalize([g, g.bfloat16()])
    with pytest.raises(ValueError):
        muon.orthogonalize(g, hold="two")
    with pytest.raises(ValueError):
        muon.orthogonalize(g, coeffs=[(1, 0, 0)])              # one triple for five steps
    with pytest.raises(ValueError):
        muon.update([g], [g], [g], lr=0.1, scale="wide")
    with pytest.raises(ValueError):
        muon.update([g], [g], [], lr=0.1)
    with pytest.raises(ValueError):
        muon.update([g], [g], [torch.zeros(4, 3)], lr=0.1)
    with pytest.raises(ValueError):
        muon.matrices([torch.zeros(3)], [torch.zeros(3)])


def test_batches_become_records():
    g = torch.zeros(2, 3, 10, 8)[:, ::2, 1:, :6]
    r = muon.matrices([g], [torch.zeros(2, 2, 9, 6)])
    assert len(r) == 4 and set(r["rows"]) == {9} and set(r["cols"]) == {6} and set(r["ld_grad"]) == {8}
    want = [g[i, j].data_ptr() for i in range(2) for j in range(2)]
    assert list(r["grad"]) == want
    assert len(muon.matrices([torch.zeros(0, 3, 4)], [torch.zeros(0, 3, 4)])) == 0


def test_deferred_micro_batches_are_closed_before_a_reduce():
    d = deferred.DeferredReducer(2, 40, device="cpu")
    with pytest.raises(RuntimeError):
        d.end_micro_batch()
    w, x, dy = torch.zeros(4, 5), torch.zeros(3, 5), torch.zeros(3, 4)
    for row, off, boff in [(2, 0, None), (-1, 0, None), (0, 21, None), (0, -1, None), (0, 0, 37), (0, 0, 19)]:
        with pytest.raises(ValueError):
            d.accumulate_linear(row, off, dy, x, w, bias_offset=boff)
    d.open = True
    for call in (lambda: d.reduce(None, 0), lambda: d.accumulate(None, 0), d.state_dict):
        with pytest.raises(RuntimeError):
            call()

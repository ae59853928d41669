"""The embedding's entry points on the host (no GPU): refusals and
workspaces."""
import pytest
import torch

from gradient_reduction_amd import dc, deferred, embedding
from tests.test_abi import FAKE, expect

FAR = 1 << 36


def at(k):
    return FAKE + k * FAR


LOOKUP = dict(dtype=0, id_bytes=8, T=4, rows=6, D=5, ids=at(0), table=at(1), ld_table=5, scale=1.0, out=at(2),
              ld_out=5, stream=0)


@pytest.mark.parametrize("code, change", [
    (dc.DC_ERR_DTYPE, dict(dtype=2)), (dc.DC_ERR_DTYPE, dict(id_bytes=2)), (dc.DC_ERR_ARG, dict(T=-1)),
    (dc.DC_ERR_ARG, dict(rows=0)), (dc.DC_ERR_ARG, dict(D=0)), (dc.DC_ERR_SHAPE, dict(T=(1 << 26) + 1)),
    (dc.DC_ERR_SHAPE, dict(D=(1 << 22) + 1)), (dc.DC_ERR_SHAPE, dict(rows=(1 << 28) + 1)),
    (dc.DC_ERR_SHAPE, dict(rows=1 << 27, D=1 << 10)), (dc.DC_ERR_ARG, dict(scale=float("nan"))),
    (dc.DC_ERR_ARG, dict(scale=float("inf"))), (dc.DC_ERR_NULL, dict(ids=None)), (dc.DC_ERR_NULL, dict(table=None)),
    (dc.DC_ERR_NULL, dict(out=None)), (dc.DC_ERR_ALIGN, dict(ids=at(0) + 4)), (dc.DC_ERR_ALIGN, dict(table=at(1) + 1)),
    (dc.DC_ERR_SHAPE, dict(ld_table=4)), (dc.DC_ERR_SHAPE, dict(ld_out=4)), (dc.DC_ERR_ARG, dict(out=at(1) + 58)),
    (dc.DC_ERR_ARG, dict(out=at(0) + 30)),
])
def test_lookup_refusals(code, change):
    expect(code, dc.dc_embedding, **{**LOOKUP, **change})


BACK = dict(dtype=0, id_bytes=4, T=4, rows=6, D=5, dy=at(0), ld_dy=5, ids=at(1), scale=1.0, grad_dtype=1,
            dtable=at(2), ld=5, accumulate=1, workspace=at(3), workspace_bytes=1 << 30, stream=0)


@pytest.mark.parametrize("code, change", [
    (dc.DC_ERR_DTYPE, dict(dtype=3)), (dc.DC_ERR_DTYPE, dict(id_bytes=0)), (dc.DC_ERR_DTYPE, dict(grad_dtype=2)),
    (dc.DC_ERR_DTYPE, dict(dtype=1, grad_dtype=0)), (dc.DC_ERR_ARG, dict(accumulate=2)), (dc.DC_ERR_ARG, dict(T=-1)),
    (dc.DC_ERR_SHAPE, dict(T=(1 << 26) + 1)), (dc.DC_ERR_ARG, dict(scale=float("nan"))), (dc.DC_ERR_NULL, dict(ids=None)),
    (dc.DC_ERR_NULL, dict(dy=None)), (dc.DC_ERR_NULL, dict(dtable=None)), (dc.DC_ERR_NULL, dict(T=0, dtable=None)),
    (dc.DC_ERR_SHAPE, dict(ld=4)), (dc.DC_ERR_SHAPE, dict(ld_dy=4)), (dc.DC_ERR_ALIGN, dict(dtable=at(2) + 2)),
    (dc.DC_ERR_ALIGN, dict(ids=at(1) + 2)), (dc.DC_ERR_ARG, dict(dtable=at(0) + 36)), (dc.DC_ERR_ARG, dict(dtable=at(1) + 4)),
    (dc.DC_ERR_SHAPE, dict(workspace_bytes=63)), (dc.DC_ERR_NULL, dict(workspace=None)),
    (dc.DC_ERR_ALIGN, dict(workspace=at(3) + 8)),
])
def test_gradient_refusals(code, change):
    expect(code, dc.dc_embedding_backward, **{**BACK, **change})


def test_workspaces():
    need = dc.dc_embedding_backward_workspace
    assert need(0, 0, 5, 5) == 0 and need(0, 1, 5, 5) % 16 == 0 and need(0, 40000, 5, 64) >= 40000 * 16
    assert need(0, 40000, 5, 128) > need(0, 40000, 5, 64)
    expect(dc.DC_ERR_NULL, lambda: dc._check("q", dc.lib().dc_embedding_backward_workspace(0, 1, 1, 1, None)))
    for bad in ((2, 1, 1, 1), (0, -1, 1, 1), (0, 1, 0, 1), (0, 1, 1, 0)):
        with pytest.raises(dc.DCError):
            need(*bad)


def test_python_refusals():
    ids, table = torch.zeros(4, dtype=torch.int64), torch.zeros(6, 5)
    for a in ((ids, table), (ids.float(), table), (ids.short(), table), (ids, table[0]), (ids, table.half()),
              (ids, table.t()[:5])):
        with pytest.raises(ValueError):
            embedding.forward(*a)
    with pytest.raises(ValueError):
        embedding.forward(ids, table, scale=float("inf"))
    dy = torch.zeros(4, 5)
    for kw in (dict(), dict(rows=6), dict(rows=6, accumulate=True), dict(dtable=table[0]), dict(dtable=table.half()),
               dict(dtable=table, scale=1e39)):
        with pytest.raises(ValueError):
            embedding.backward(dy, ids, **kw)


def test_refused_before_anything_is_launched(monkeypatch):
    """What a refused layer leaves of the accumulators, without a GPU."""
    import contextlib
    from gradient_reduction_amd import linear
    seen = []
    monkeypatch.setattr(linear, "on", lambda device, stream: contextlib.nullcontext())
    monkeypatch.setattr(dc, "dc_embedding_backward", lambda *a: seen.append(a))
    d = deferred.DeferredReducer(2, 100, device="cpu")
    d.acc.fill_(7.0)
    ids, dy = torch.zeros(4, dtype=torch.int64), torch.zeros(4, 5)
    over = torch.as_strided(d.acc, (4, 5), (5, 1), 20)
    for kw in (dict(row=2), dict(offset=80), dict(dy=dy[:3]), dict(ids=ids.float()), dict(dy=over), dict(scale=1e39),
               dict(dy=dy.double())):
        with pytest.raises(ValueError):
            d.accumulate_embedding(**{**dict(row=0, offset=3, dy=dy, ids=ids, rows=6), **kw})
        assert not seen and bool((d.acc == 7).all()) and not d.open
    d.accumulate_embedding(0, 3, dy, ids, 6)
    assert len(seen) == 1 and d.open and not d.acc[0].any() and bool((d.acc[1] == 7).all())


def test_a_gradient_without_columns_is_refused():
    d = deferred.DeferredReducer(2, 100, device="cpu")
    ids = torch.zeros((), dtype=torch.int64)
    for rows in (6, 0, -1):
        with pytest.raises(ValueError):
            d.accumulate_embedding(0, 3, torch.zeros(()), ids, rows)
    for rows in (0, -1):
        with pytest.raises(ValueError):
            d.accumulate_embedding(0, 3, torch.zeros(4, 5), torch.zeros(4, dtype=torch.int64), rows)
        with pytest.raises(ValueError):
            embedding.backward(torch.zeros(4, 5), torch.zeros(4, dtype=torch.int64), rows=rows)

"""What a layer's backward refuses, and when (no GPU): launches are replaced
by a record of them, and every refusal comes before the first."""
import contextlib
import random

import numpy as np
import pytest
import torch

from gradient_reduction_amd import dc, deferred, linear

T, N, K = 3, 4, 5


@pytest.fixture
def launches(monkeypatch):
    seen = []
    monkeypatch.setattr(linear, "on", lambda device, stream: contextlib.nullcontext())
    for name in ("dc_bias_act_backward", "dc_linear_backward"):
        monkeypatch.setattr(dc, name, lambda *a, name=name: seen.append(name))
    return seen


def operands():
    return {"dy": torch.zeros(T, N), "x": torch.zeros(T, K), "w": torch.zeros(N, K), "pre": torch.zeros(T, N)}


def call(o, act="gelu", **kw):
    return linear.backward(o["dy"], o["x"], o["w"], o["pre"], act, accumulate=True, **kw)


def inside(t, at, *shape):
    """A tensor of `shape` over the elements of t's storage from `at` on."""
    n = 1
    for s in shape:
        n *= s
    return torch.as_strided(t, shape, (shape[-1], 1) if len(shape) == 2 else (1,), at) if n + at <= t.numel() else None


@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("name", ["dy", "x", "w", "pre", "dw"])
def test_a_bias_gradient_over_another_operand(launches, name, act):
    if (name, act) == ("pre", "none"):
        return                # not read
    o = operands()
    dw = torch.zeros(N, K)
    over = dw if name == "dw" else o[name]
    for at in (0, over.numel() - N):
        with pytest.raises(ValueError, match="db"):
            call(o, act=act, dw=dw, db=inside(over, at, N))
        assert not launches
        if name in ("dy", "w", "pre"):     # without a weight gradient too: then x is not read
            with pytest.raises(ValueError, match="db"):
                call(o, act=act, db=inside(over, at, N), need_dw=False)
            assert not launches


@pytest.mark.parametrize("act, name", [("gelu", "x"), ("gelu", "w"), ("none", "dy"), ("none", "x")])
def test_a_weight_gradient_over_another_operand(launches, act, name):
    flat = torch.zeros(100)
    o = operands()
    rows, cols = o[name].shape
    o[name] = flat[30:30 + rows * cols].view(rows, cols)
    for at in (30, 30 + rows * cols - 1, 31 - N * K):
        with pytest.raises(ValueError, match="dw"):
            call(o, act=act, dw=flat[at:at + N * K].view(N, K), db=torch.zeros(N))
        assert not launches
    # next to it
    for at in (30 + rows * cols, 30 - N * K):
        call(o, act=act, dw=flat[at:at + N * K].view(N, K), db=torch.zeros(N))
    assert launches == ["dc_bias_act_backward", "dc_linear_backward"] * 2


def test_interleaved_columns_are_apart(launches):
    wide = torch.zeros(N, 2 * K + 1)
    o = operands()
    o["w"] = wide[:, :K]
    call(o, dw=wide[:, K:2 * K], db=torch.zeros(N))
    assert len(launches) == 2
    with pytest.raises(ValueError, match="dw"):
        call(o, dw=wide[:, K - 1:2 * K - 1], db=torch.zeros(N))
    assert len(launches) == 2


def test_gradients_where_nothing_is_read_any_more(launches):
    """Between another operand's rows; over dy and pre, which the elementwise
    part has read; over x or w, where the other gradient alone is made."""
    o = operands()
    wide = torch.zeros(N, K + N)
    call(o, dw=wide[:, :K], db=wide[0, K:])
    call(o, dw=wide[:, :K], db=wide[N - 2, K:])
    for at in (K - 1, K + 1):       # wide's elements K - 1 and K + N
        with pytest.raises(ValueError, match="db"):
            call(o, dw=wide[:, :K], db=wide.view(-1)[at:at + N])
    flat = torch.zeros(100)
    o["dy"], o["pre"] = flat[:T * N].view(T, N), flat[50:50 + T * N].view(T, N)
    call(o, dw=flat[:N * K].view(N, K))
    call(o, dw=flat[45:45 + N * K].view(N, K))
    o = operands()
    call(o, dw=o["w"], need_dx=False)
    call(o, db=o["x"].view(-1)[:N], need_dw=False)
    assert launches.count("dc_linear_backward") == 6


def test_refusals_of_any_kind_come_first(launches, monkeypatch):
    o = operands()
    db, dw = torch.zeros(N), torch.zeros(N, K)
    for change, kw in [({"pre": None}, {}), ({"pre": torch.zeros(T, N + 1)}, {}), ({"pre": torch.zeros(T + 1, N)}, {}),
                       ({"dy": torch.zeros(T, N + 1)}, {}), ({"x": torch.zeros(T, 0), "w": torch.zeros(N, 0)}, {}),
                       ({}, {"db": torch.zeros(N + 1)}), ({}, {"db": torch.zeros(N).double()}),
                       ({}, {"dw": torch.zeros(N, K).double()}), ({}, {"dw": torch.zeros(K, N)}), ({}, {"act": "tanh"})]:
        args = {"db": db, "dw": dw, **kw}
        if "x" in change:
            args["dw"] = torch.zeros(N, 0)
        with pytest.raises((ValueError, dc.DCError)):
            call({**o, **change}, **args)
        assert not launches, (change, kw)

    def full(*a, **k):
        raise MemoryError

    monkeypatch.setattr(linear, "workspace", full)       # no memory is left
    with pytest.raises(MemoryError):
        call(o, db=db, dw=dw)
    assert not launches


def test_a_refused_layer_leaves_the_accumulators(launches):
    """What reduce(keep_acc=True) or anything else left in them stays until a
    layer is accepted."""
    red = deferred.DeferredReducer(2, 40, device="cpu")
    red.acc.fill_(7.0)
    o = operands()
    for change, kw in [({"pre": None}, {}), ({"pre": torch.zeros(T, N + 1)}, {}), ({"dy": torch.zeros(T, N + 1)}, {}),
                       ({"x": torch.zeros(T, K).double()}, {}), ({}, {"act": "tanh"}),
                       ({"x": red.acc[0, :T * K].view(T, K)}, {}), ({"dy": red.acc[0, 20:20 + T * N].view(T, N)}, {})]:
        a = {**o, **change}
        with pytest.raises(ValueError):
            red.accumulate_linear(0, 0, a["dy"], a["x"], a["w"], a["pre"], **{"act": "gelu", "bias_offset": 20, **kw})
        assert not launches and not red.open and bool((red.acc == 7).all()), change
    red.accumulate_linear(0, 0, o["dy"], o["x"], o["w"], o["pre"], act="gelu", bias_offset=20)
    assert launches and red.open and bool((red.acc[0] == 0).all())


def test_a_layer_touches_its_own_replicas_accumulators_only(launches, monkeypatch):
    """Replicas may be on streams of their own, so a layer of one may not clear
    another's row: each row is cleared by its replica's first layer of the step,
    and one without any before the row is next used."""
    red = deferred.DeferredReducer(3, 40, device="cpu")
    o = operands()

    def add(row):
        red.accumulate_linear(row, 0, o["dy"], o["x"], o["w"])
        red.acc[row, 3] += 1.0          # as the product would

    def rows():
        return [red.acc[r, 3].item() for r in range(3)]

    monkeypatch.setattr(dc, "dc_deferred_reduce", lambda *a: None)
    monkeypatch.setattr(dc, "dc_accumulate", lambda *a: red.acc.add_(10.0) if a[-2] == 0 else red.acc.fill_(10.0))
    red.acc.fill_(7.0)
    add(1)
    assert rows() == [7, 1, 7]
    add(0)
    add(1)
    assert rows() == [1, 2, 7]
    red.end_micro_batch()
    add(0)
    red.end_micro_batch()
    assert rows() == [2, 2, 7]
    assert red.state_dict()["acc"][:, 3].tolist() == [2, 2, 0] and rows() == [2, 2, 0]
    red.reduce(None, 0)
    # a step whose second micro-batch comes whole
    red.acc.fill_(7.0)
    add(2)
    red.end_micro_batch()
    red.accumulate(None, 0)
    assert rows() == [10, 10, 11]
    red.reduce(None, 0)
    # one that is reduced with rows without layers
    red.acc.fill_(7.0)
    add(0)
    red.end_micro_batch()
    red.reduce(None, 0)
    assert rows() == [1, 0, 0]
    # one that is replaced by a saved state, and one of whole micro-batches
    add(0)
    red.load_state_dict({"acc": torch.full((3, 40), 5.0), "micro_batches": 1})
    add(1)
    assert rows() == [5, 6, 5]
    red.end_micro_batch()
    red.reduce(None, 0)
    red.accumulate(None, 0)
    assert rows() == [10, 10, 10]


def elements(at, rows, cols, ld):
    return {at + r * ld + c for r in range(rows) for c in range(cols)}


def test_overlap_is_found_exactly():
    """The library's check and the one before it against the elements
    themselves: exact for rows of one stride and for a single row; matrices of
    different strides may not interleave."""
    rng = random.Random(5)
    flat = torch.zeros(400)
    base, far = 1 << 32, 1 << 40
    coeffs = np.tile(np.array([3.4445, -4.775, 2.0315], np.float32), (5, 1))
    seen = set()
    for _ in range(4000):
        a, b = [(rng.randrange(60), rng.choice([1, 1, 2, 3, 4]), rng.randint(1, 6)) for _ in range(2)]
        ld = [v[2] + rng.randrange(9) for v in (a, b)]
        if rng.random() < 0.5:
            ld = [max(ld)] * 2
        ea, eb = elements(*a, ld[0]), elements(*b, ld[1])
        want = bool(ea & eb)
        if a[1] > 1 and b[1] > 1 and ld[0] != ld[1]:
            want = max(ea) >= min(eb) and max(eb) >= min(ea)
        views = [torch.as_strided(flat, v[1:], (d, 1), v[0]) for v, d in ((a, ld[0]), (b, ld[1]))]
        spans = [linear._span("ab"[k], t, *v[1:], d, 4) for k, (t, v, d) in enumerate(zip(views, (a, b), ld))]
        with pytest.raises(ValueError, match="a and b overlap") if want else contextlib.nullcontext():
            linear._apart(spans[0], spans[1:])
        m = np.zeros(2, dc.MATRIX_DTYPE)
        m["rows"], m["cols"] = (a[1], b[1]), (a[2], b[2])
        m["out"], m["ld_out"] = (base + 4 * a[0], far), (ld[0], b[2])
        m["grad"], m["ld_grad"] = (2 * far, base + 4 * b[0]), (a[2], ld[1])
        with pytest.raises(dc.DCError) as e:       # the workspace is too small
            dc.dc_orthogonalize(dc.DC_F32, 0, m, 2, 5, coeffs, 1e-7, 3 * far, 16, 0)
        assert ("overlap" in str(e.value)) == want, (a, b, ld, e.value)
        seen.add((want, a[1] == 1, b[1] == 1, ld[0] == ld[1]))
    assert len(seen) == 16

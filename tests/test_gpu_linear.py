"""The linear layer's products on the GPU against their definition in 64 bits.

Bounds, elementwise.  Inputs are exact in their dtype.  A sum of K products in
fp32 rounds (or, inside a matrix instruction, truncates) K products and K adds
at most, each by a step 2^-23 of what is added up, so it is off by at most
2 K 2^-23 S with S = sum |x| |w|; the bias and the joining of split sums add a
few.  Activations have slopes of at most 1.13 and are computed to 2^-20 of
their argument's size; the result is rounded once to the dtype, by
finfo.eps / 2 of its value."""
import numpy as np
import pytest

from gradient_reduction_amd import dc, deferred, executor, linear, muon

pytestmark = pytest.mark.gpu
STEP = 2.0 ** -23


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    import torch
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    dc.lib()
    yield
    torch.cuda.synchronize()


def T():
    import torch
    return torch


def dt(name):
    return T().bfloat16 if name == "bf16" else T().float32


def half_step(name):
    return T().finfo(dt(name)).eps / 2


def randn(gen, *shape, scale=1.0, dtype=None, pad=0, shift=0):
    """A [.., cols] tensor; with pad, rows that many elements apart from NaNs;
    with shift, a base that is not 16-byte aligned."""
    t = T()
    v = (t.randn(*shape, generator=gen, dtype=t.float64) * scale).to(dtype)
    if not pad and not shift:
        return v.cuda()
    rows, cols = shape
    flat = t.full((rows * (cols + pad) + shift,), float("nan"), dtype=dtype, device="cuda")
    out = flat[shift:].view(rows, cols + pad)[:, :cols]
    out.copy_(v)
    return out


def act64(v, act):
    t = T()
    if act == "relu":
        return t.clamp(v, min=0)
    if act == "gelu":
        return v * t.special.ndtr(v)
    if act == "silu":
        return v * t.special.expit(v)
    return v


def slope64(v, act):
    t = T()
    if act == "relu":
        return (v > 0).double()
    if act == "gelu":
        return t.special.ndtr(v) + v * t.exp(-v * v / 2) / (2 * np.pi) ** 0.5
    if act == "silu":
        p = t.special.expit(v)
        return p * (1 + v * (1 - p))
    return t.ones_like(v)


def host(*xs):
    return [None if x is None else x.detach().cpu().double() for x in xs]


def inside(name, got, want, bound):
    t = T()
    got = got.cpu().double()
    assert bool(t.isfinite(got).all()), f"{name}: not finite"
    off = ((got - want).abs() - bound).max().item() if got.numel() else -1.0
    assert off <= 0, f"{name}: {off:.3g} over the bound, at {((got - want).abs() - bound).argmax().item()}"


SIZES = [(1, 1, 1), (1, 16, 8), (3, 5, 7), (2, 700, 4096), (5, 1003, 515), (16, 64, 64), (17, 130, 65), (31, 33, 1),
         (64, 64, 64), (100, 129, 257), (128, 128, 128), (129, 256, 72), (200, 96, 1000), (64, 72, 8192),
         (257, 300, 520), (515, 1, 130), (1, 1, 9000), (700, 513, 64)]


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_forward(size, kind):
    t = T()
    rows, n, k = size
    gen = t.Generator().manual_seed(rows * 1000003 + n * 1009 + k)
    h, eps = dt(kind), half_step(kind)
    for variant, (act, with_bias, with_res, pad, shift) in enumerate([
            ("none", False, False, 0, 0), ("gelu", True, True, 0, 0), ("silu", True, False, 8, 0),
            ("relu", False, True, 3, 1), ("gelu", True, True, 0, 1)]):
        x = randn(gen, rows, k, dtype=h, pad=pad, shift=shift)
        w = randn(gen, n, k, scale=k ** -0.5, dtype=h, pad=pad, shift=shift)
        b = randn(gen, n, dtype=h) if with_bias else None
        r = randn(gen, rows, n, dtype=h, pad=pad, shift=shift) if with_res else None
        out = t.full((rows, n + pad), 7.0, dtype=h, device="cuda")
        pre = t.full((rows, n + pad), 7.0, dtype=h, device="cuda")
        y, z = linear.forward(x, w, b, r, act=act, out=out[:, :n], pre=pre[:, :n])
        plain = linear.forward(x, w, b, r, act=act)
        assert t.equal(plain, y), f"variant {variant}: saving pre changes y"
        if pad:
            assert bool((out[:, n:] == 7).all()) and bool((pre[:, n:] == 7).all())
        hx, hw, hb, hr = host(x, w, b, r)
        want = hx @ hw.t()
        s = hx.abs() @ hw.abs().t()
        if hb is not None:
            want, s = want + hb, s + hb.abs()
        sums = (2 * k + 8) * STEP * s
        inside(f"pre {variant}", z, want, sums + eps * (want.abs() + sums))
        a = act64(want, act)
        total = a if hr is None else a + hr
        err = 1.13 * sums + 2.0 ** -20 * (want.abs() + a.abs())
        err = err + 2 * STEP * (a.abs() + total.abs())
        inside(f"y {variant}", y, total, err + eps * (total.abs() + err))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_forward_in_place_and_empty(kind):
    t = T()
    gen = t.Generator().manual_seed(5)
    x, w = randn(gen, 70, 96, dtype=dt(kind)), randn(gen, 130, 96, dtype=dt(kind))
    r = randn(gen, 70, 130, dtype=dt(kind))
    want = linear.forward(x, w, residual=r.clone(), act="silu")
    got = linear.forward(x, w, residual=r, act="silu", out=r)
    assert got.data_ptr() == r.data_ptr() and t.equal(got, want)
    assert linear.forward(x[:0], w).shape == (0, 130)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_one_bad_row_stays_in_its_row(kind):
    """NaN and infinity in one token's input reach that token's outputs only."""
    t = T()
    gen = t.Generator().manual_seed(6)
    for rows in (3, 40, 200):
        x, w = randn(gen, rows, 100, dtype=dt(kind)), randn(gen, 90, 100, dtype=dt(kind))
        clean = linear.forward(x, w)
        bad = x.clone()
        bad[1, 7], bad[2, 99] = float("nan"), float("inf")
        y = linear.forward(bad, w)
        assert bool(t.isnan(y[1]).all()) and not bool(t.isfinite(y[2]).any())
        keep = [i for i in range(rows) if i not in (1, 2)]
        assert t.equal(y[keep], clean[keep])


@pytest.mark.parametrize("kind, grad", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("size", [(0, 5, 6), (1, 1, 1), (1, 40, 300), (3, 5, 7), (17, 130, 65), (64, 64, 64), (100, 129, 257),
                                  (128, 128, 128), (300, 96, 72), (257, 300, 520), (8192, 72, 64), (1000, 16, 8),
                                  (5, 1003, 515)], ids=str)
def test_backward_products(size, kind, grad):
    t = T()
    rows, n, k = size
    gen = t.Generator().manual_seed(rows * 7 + n * 31 + k)
    h, g = dt(kind), dt(grad)
    for variant, (acc, pad, shift) in enumerate([(False, 0, 0), (True, 0, 0), (True, 8, 0), (False, 3, 1)]):
        dy = randn(gen, rows, n, dtype=h, pad=pad, shift=shift)
        x = randn(gen, rows, k, dtype=h, pad=pad, shift=shift)
        w = randn(gen, n, k, dtype=h, pad=pad, shift=shift)
        dw0, db0 = randn(gen, n, k, dtype=g), randn(gen, n, dtype=g)
        hold = t.full((n, k + pad), 7.0, dtype=g, device="cuda")
        dw, db = hold[:, :k], db0.clone()
        dw.copy_(dw0)
        dx, dw2, db2 = linear.backward(dy, x, w, dw=dw, db=db, accumulate=acc)
        assert dw2.data_ptr() == dw.data_ptr() and db2.data_ptr() == db.data_ptr()
        if pad:
            assert bool((hold[:, k:] == 7).all())
        hy, hx, hw, hdw, hdb = host(dy, x, w, dw0, db0)
        want, s = hy @ hw, hy.abs() @ hw.abs()
        sums = (2 * n + 8) * STEP * s
        inside(f"dx {variant}", dx, want, sums + half_step(kind) * (want.abs() + sums))
        for name, got, v, s in (("dw", dw, hy.t() @ hx + acc * hdw, hy.abs().t() @ hx.abs() + acc * hdw.abs()),
                                ("db", db, hy.sum(0) + acc * hdb, hy.abs().sum(0) + acc * hdb.abs())):
            sums = (2 * rows + 8) * STEP * s
            inside(f"{name} {variant}", got, v, sums + half_step(grad) * (v.abs() + sums))
    if rows:
        only, none, _ = linear.backward(dy, x, w, need_dw=False)
        assert none is None and t.equal(only, dx)
        none, dw3, _ = linear.backward(dy, x, w, need_dx=False, grad_dtype=g)
        assert none is None and t.equal(dw3, dw)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["none", "relu", "gelu", "silu"])
@pytest.mark.parametrize("size", [(0, 9), (1, 1), (1, 700), (3, 9), (33, 256), (333, 1003), (5000, 40)], ids=str)
def test_bias_act_backward(size, act, kind):
    t = T()
    rows, n = size
    gen = t.Generator().manual_seed(rows + 17 * n)
    h = dt(kind)
    for variant, (acc, pad, shift, grad) in enumerate([(False, 0, 0, "f32"), (True, 8, 0, kind), (True, 3, 1, "f32")]):
        dy = randn(gen, rows, n, dtype=h, pad=pad, shift=shift)
        pre = randn(gen, rows, n, scale=2.0, dtype=h, pad=pad, shift=shift)
        db0 = randn(gen, n, dtype=dt(grad))
        db = db0.clone()
        hold = t.full((rows, n + pad), 7.0, dtype=h, device="cuda")
        dz, db2 = linear.bias_act_backward(dy, pre, act, dz=hold[:, :n], db=db, accumulate=acc)
        assert db2.data_ptr() == db.data_ptr()
        if pad:
            assert bool((hold[:, n:] == 7).all())
        hy, hp, hb = host(dy, pre, db0)
        want = hy * slope64(hp, act)
        # the slope: of size <= 1.13, computed to 2^-20; then the product
        err = 2.0 ** -19 * hy.abs()
        inside(f"dz {variant}", dz, want, err + half_step(kind) * (want.abs() + err))
        sums = err.sum(0) + (rows + 8) * STEP * (1.13 * hy.abs().sum(0) + acc * hb.abs())
        v = want.sum(0) + acc * hb
        inside(f"db {variant}", db, v, sums + half_step(grad) * (v.abs() + sums))
        alone, _ = linear.bias_act_backward(dy, pre, act)
        assert t.equal(alone, dz)
    if act != "none":
        same = dy.clone()
        z, _ = linear.bias_act_backward(same, pre, act, dz=same)
        assert t.equal(z, dz)


@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
def test_gradients_match_differences(act):
    """Central differences of the definition in 64 bits, step 1e-4: off by
    1e-8 of third derivatives (under 5 here) and 1e-12 of rounding, beside the
    fp32 gradients' 2^-18 of the sums' size."""
    t = T()
    gen = t.Generator().manual_seed(11)
    rows, n, k = 9, 13, 21
    x, w, b = (randn(gen, rows, k, dtype=t.float32), randn(gen, n, k, scale=0.3, dtype=t.float32),
               randn(gen, n, dtype=t.float32))
    dy = randn(gen, rows, n, dtype=t.float32)
    _, pre = linear.forward(x, w, b, act=act, save_pre=True)
    db = t.zeros(n, device="cuda")
    dx, dw, db = linear.backward(dy, x, w, pre, act, db=db)
    hx, hw, hb, hy = host(x, w, b, dy)

    def loss(x, w, b):
        return (hy * act64(x @ w.t() + b, act)).sum()

    for got, at in ((dx, 0), (dw, 1), (db, 2)):
        args = [hx, hw, hb]
        base = args[at]
        for i in list(range(0, base.numel(), 7)):
            e = t.zeros(base.numel(), dtype=t.float64)
            e[i] = 1e-4
            e = e.view(base.shape)
            up, down = list(args), list(args)
            up[at], down[at] = base + e, base - e
            d = (loss(*up) - loss(*down)) / 2e-4
            size = hy.abs().sum().item() * max(1.0, hx.abs().max().item())
            assert abs(got.cpu().view(-1)[i].item() - d.item()) < (1e-7 + 2.0 ** -18) * size


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["relu", "gelu", "silu"])
@pytest.mark.parametrize("rows", [1, 70])
def test_values_of_any_size(rows, act, kind):
    """Activations and slopes where exp(-v), exp(-v^2 / 2) or v^2 leave fp32's
    range.  Those values are exact: v or 0, and slopes 1 or 0 (within 1e-35 from
    |v| = 100 on); infinity gives infinity, NaN NaN."""
    t = T()
    sizes = t.tensor([100.0, 2.0 ** 10, 2.0 ** 40, 2.0 ** 63, 2.0 ** 64, 2.0 ** 65, 2.0 ** 100, 2.0 ** 127, 3.3e38],
                     dtype=t.float32)
    v = t.cat([sizes, -sizes]).to(dt(kind))
    n = v.numel()
    x = t.ones(rows, 1, dtype=dt(kind), device="cuda")
    y = linear.forward(x, v.view(n, 1).cuda(), act=act)
    want = t.where(v > 0, v, t.zeros_like(v)).double().expand(rows, n)
    assert (host(y)[0] - want).abs().max() <= 1e-35
    pre = v.expand(rows, n).contiguous().cuda()
    dz, _ = linear.bias_act_backward(t.ones_like(pre), pre, act=act)
    assert (host(dz)[0] - (v > 0).double().expand(rows, n)).abs().max() <= 1e-35
    odd = t.tensor([[float("inf")], [float("nan")]], dtype=dt(kind), device="cuda")
    y = host(linear.forward(x, odd, act=act))[0]
    assert (y[:, 0] == float("inf")).all() and y[:, 1].isnan().all()


def test_few_rows_of_many_outputs():
    """More outputs than the few-row kernel's grid takes: small whole numbers,
    so the sums are exact in any order."""
    t = T()
    n, k = 2 ** 26 + 24, 8
    w = t.randint(-4, 5, (n, k), dtype=t.int8, device="cuda").bfloat16()
    x = t.randint(-4, 5, (2, k), dtype=t.int8, device="cuda").bfloat16()
    y = linear.forward(x, w)
    for at in range(0, n, 2 ** 24):
        part = w[at:at + 2 ** 24].float()
        for i in range(2):
            assert t.equal(y[i, at:at + 2 ** 24].float(), (part * x[i].float()).sum(1))


def layer(t, gen, rows, n, k, kind):
    h = dt(kind)
    return (randn(gen, rows, k, dtype=h), randn(gen, n, k, scale=k ** -0.5, dtype=h), randn(gen, n, dtype=h),
            randn(gen, rows, n, dtype=h))


def whole(x, w, b, dy, dw, db):
    y, pre = linear.forward(x, w, b, act="gelu", save_pre=True)
    return (y, pre) + linear.backward(dy, x, w, pre, "gelu", dw=dw, db=db, accumulate=True)


@pytest.mark.parametrize("size", [(1, 512, 256), (70, 100, 3000), (300, 257, 130)], ids=str)
def test_replayed_and_on_other_streams(size):
    """A recorded layer, replayed with other inputs and eager work between,
    and two layers at once on two streams, give the eager results bit for
    bit."""
    t = T()
    gen = t.Generator().manual_seed(3)
    sets = [layer(t, gen, *size, "bf16") for _ in range(3)]
    rows, n, k = size

    def grads():
        return t.ones(n, k, device="cuda"), t.ones(n, device="cuda")

    eager = [whole(*s, *grads()) for s in sets]
    t.cuda.synchronize()
    static = [v.clone() for v in sets[0]]
    dw, db = grads()
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        rec = whole(*static, dw, db)
    for s, want in list(zip(sets, eager)) * 2:
        for a, b in zip(static, s):
            a.copy_(b)
        dw.fill_(1.0)
        db.fill_(1.0)
        g.replay()
        whole(*s, *grads())
        t.cuda.synchronize()
        for a, b in zip(rec, want):
            assert t.equal(a, b)
    streams = [t.cuda.Stream() for _ in range(2)]
    outs = []
    for rep in range(3):
        for s, st in zip(sets, streams):
            st.wait_stream(t.cuda.current_stream())
            y, pre = linear.forward(s[0], s[1], s[2], act="gelu", save_pre=True, stream=st)
            with t.cuda.stream(st):
                d = grads()
            outs.append((y, pre) + linear.backward(s[3], s[0], s[1], pre, "gelu", dw=d[0], db=d[1],
                                                   accumulate=True, stream=st.cuda_stream))
    t.cuda.synchronize()
    for i, o in enumerate(outs):
        for a, b in zip(o, eager[i % 2]):
            assert t.equal(a, b)


def test_offsets_past_32_bits():
    """Rows of an operand more than 2^31 elements apart from its base."""
    t = T()
    ld = (1 << 25) + 40
    rows = 70
    big = t.empty(rows * ld, dtype=t.bfloat16, device="cuda")
    x = big.view(rows, ld)[:, 11:11 + 96]
    gen = t.Generator().manual_seed(9)
    x.copy_(randn(gen, rows, 96, dtype=t.bfloat16))
    w, dy = randn(gen, 50, 96, dtype=t.bfloat16), randn(gen, rows, 50, dtype=t.bfloat16)
    near = x.contiguous()
    assert t.equal(linear.forward(x, w), linear.forward(near, w))
    aligned = big.view(rows, ld)[:, 16:16 + 96]
    keep = near.clone()
    aligned.copy_(keep)
    assert t.equal(linear.forward(aligned, w), linear.forward(near, w))
    out = big.view(rows, ld)[:, 200:250]
    assert t.equal(linear.forward(near, w, out=out), linear.forward(near, w))
    for a, b in zip(linear.backward(dy, aligned, w), linear.backward(dy, near, w)):
        assert b is None or t.equal(a, b)


def test_layers_into_the_deferred_reduction():
    """Two replicas, three micro-batches, two layers and one weight used
    twice: the products' sums in the accumulators, reduced, against the
    definition in 64 bits; and the same sums through the micro-batch slabs."""
    t = T()
    W, rows, n, k = 2, 50, 24, 40
    offs = {"w1": 3, "b1": 3 + n * k, "w2": 3 + n * k + n}       # odd places
    M = offs["w2"] + k * n
    red = deferred.DeferredReducer(W, M)
    slab = deferred.DeferredReducer(W, M)
    gen = t.Generator().manual_seed(21)
    h = t.bfloat16
    want = t.zeros(M, dtype=t.float64)
    size = t.zeros(M, dtype=t.float64)
    w1, b1, w2 = randn(gen, n, k, scale=k ** -0.5, dtype=h), randn(gen, n, dtype=h), randn(gen, k, n, scale=n ** -0.5, dtype=h)
    for rep in range(2):                    # the second step must not see the first
        want.zero_()
        size.zero_()
        for mb in range(3):
            micro = t.zeros(W, red.ld, device="cuda")
            for r in range(W):
                x, dy = randn(gen, rows, k, dtype=h), randn(gen, rows, k, scale=0.1, dtype=h)
                hid, pre = linear.forward(x, w1, b1, act="silu", save_pre=True)
                dh = red.accumulate_linear(r, offs["w2"], dy, hid, w2)
                dz, db = linear.bias_act_backward(dh, pre, "silu", need_db=True)
                red.accumulate_linear(r, offs["w1"], dh, x, w1, pre, "silu", bias_offset=offs["b1"], need_dx=False)
                red.accumulate_linear(r, offs["w1"], dz, x, w1, need_dx=False)     # used twice
                hx, hdy, hh, hz = host(x, dy, hid, dz)
                parts = [(offs["w2"], hdy.t() @ hh, hdy.abs().t() @ hh.abs()),
                         (offs["w1"], 2 * hz.t() @ hx, 2 * hz.abs().t() @ hx.abs()),
                         (offs["b1"], host(db)[0], hz.abs().sum(0))]
                for o, v, s in parts:
                    want[o:o + v.numel()] += v.reshape(-1)
                    size[o:o + v.numel()] += s.reshape(-1)
                    micro[r, o:o + v.numel()] = v.reshape(-1).float().cuda()
            red.end_micro_batch()
            slab.accumulate(micro, red.ld)
        out = t.zeros(1, red.ld, device="cuda")
        other = t.zeros(1, red.ld, device="cuda")
        red.reduce(out, red.ld)
        slab.reduce(other, red.ld)
        t.cuda.synchronize()
        # 2 T roundings per product's sum and the adds of 3 micro-batches and 2 rows
        bound = (2 * rows + 16) * STEP * size
        inside("reduced", out[0, :M], want, bound)
        inside("slabs", other[0, :M], want, bound)


def test_refused_backward_leaves_db():
    t = T()
    dy, x, w = (t.ones(s, device="cuda") for s in ((4, 5), (4, 6), (5, 6)))
    for dw in (t.zeros(5, 7, device="cuda"), t.zeros(5, 6), t.zeros(5, 6, device="cuda").double()):
        db = t.zeros(5, device="cuda")
        with pytest.raises(ValueError):
            linear.backward(dy, x, w, dw=dw, db=db, accumulate=True)
        assert not db.any()

"""The norms around a block on the GPU against their definition in 64 bits.

Bounds, with h = 2^-24 (half a step of fp32, one rounding) and inputs exact in
their dtype.  1 / rms is within 4 h: the hardware's reciprocal root 2 h, its
argument's rounding h / 2.  A product of k factors rounds k - 1 times, a sum
offset + gain once.  Errors of what is computed before are carried through the
formulas' derivatives (`drift` below); a sum over T rows adds (T + 40) h of its
terms' sizes, and an output is rounded once, by half a step of its dtype."""
import pytest
import torch

from gradient_reduction_amd import dc, deferred, norm

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
H = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    dc.lib()
    yield
    torch.cuda.synchronize()


def half_step(kind):
    return torch.finfo(DT[kind]).eps / 2


def randn(gen, shape, kind, scale=1.0, mean=0.0, pad=0, shift=0):
    v = (torch.randn(shape, generator=gen, dtype=torch.float64) * scale + mean).to(DT[kind])
    if (not pad and not shift) or v.dim() != 2:
        return v.cuda()
    rows, cols = shape
    flat = torch.full((rows * (cols + pad) + shift,), float("nan"), dtype=v.dtype, device="cuda")
    out = flat[shift:].view(rows, cols + pad)[:, :cols]
    out.copy_(v)
    return out


def host(x):
    return None if x is None else x.detach().cpu().double()


def inside(name, got, want, bound):
    got = host(got)
    assert bool(torch.isfinite(got).all()), name
    off = ((got - want).abs() - bound).max().item() if got.numel() else -1.0
    assert off <= 0, f"{name}: {off:.3g} over the bound"


def gate_rows(gate, T):
    if gate is None:
        return None
    g = gate.view(-1, gate.shape[-1])
    return g.repeat_interleave(max(T // g.shape[0], 1), dim=0)[:T] if T else g[:0]


def mean(v):
    return v.mean(-1, keepdim=True)


class Case:
    """Operands of one call, and what they give in 64 bits with its bounds."""

    def __init__(self, gen, T, D, kind, post, gate, block, gain, pad=0, shift=0, scale=1.0, offset=0.0, eps=1e-6):
        self.T, self.D, self.kind, self.scale, self.offset = T, D, kind, scale, offset
        self.eps = torch.tensor(eps).item()
        about = 1.0 - offset
        self.x = randn(gen, (T, D), kind, 2.0, pad=pad, shift=shift)
        self.h = randn(gen, (T, D), kind, 0.5, pad=pad, shift=shift) if block else None
        self.post = randn(gen, (D,), kind, 0.3, about) if post else None
        self.gain = randn(gen, (D,), kind, 0.3, about) if gain else None
        self.gate = None
        if gate:
            self.gate = randn(gen, (D,) if gate == 1 else (gate, D), kind, 0.5, 0.5, pad=pad, shift=shift)
        self.dy = randn(gen, (T, D), kind, 1.0, pad=pad, shift=shift) if gain else None
        self.ds = randn(gen, (T, D), kind, 1.0, pad=pad, shift=shift)

    def kw(self):
        return dict(h=self.h, post_gain=self.post, gate=self.gate, scale=self.scale, offset=self.offset, eps=self.eps)

    def forward64(self):
        """s, its error before rounding, y, its error."""
        x, h, post, gain, gate = map(host, (self.x, self.h, self.post, self.gain, self.gate))
        scale, offset = torch.tensor(self.scale).double(), torch.tensor(self.offset).double()
        s, err = x, torch.zeros_like(x)
        if h is not None:
            u = h
            if post is not None:
                u = (offset + post) * h / (mean(h * h) + self.eps).sqrt()
            u = scale * u * (1.0 if gate is None else gate_rows(gate, self.T))
            s = x + u
            err = 9 * H * u.abs() + H * s.abs()
        if gain is None:
            return s, err, None, None
        r = 1 / (mean(s * s) + self.eps).sqrt()
        y = (offset + gain) * s * r
        drift = mean(err * err).sqrt() * r
        return s, err, y, 1.01 * ((offset + gain).abs() * r * err + y.abs() * (drift + 7 * H))

    def backward64(self, s, dgain, dpost, dgate, keep):
        """(value, bound before rounding) of dx, dh, dgain, dpost, dgate."""
        s, h, post, gain, gate, dy, ds = map(host, (s, self.h, self.post, self.gain, self.gate, self.dy, self.ds))
        scale, offset = torch.tensor(self.scale).double(), torch.tensor(self.offset).double()
        T = self.T

        def total(terms, err, old):
            v, size = terms.sum(-2), terms.abs().sum(-2)
            if old is not None and keep:
                v, size = v + host(old), size + host(old).abs()
            return v, 1.01 * (err.sum(-2) + (T + 40) * H * size)

        def through(v, g, err_g):
            r = 1 / (mean(v * v) + self.eps).sqrt()
            n = v * r
            spread = g.abs() + n.abs() * mean((g * n).abs())
            return r * (g - n * mean(g * n)), r * (err_g + n.abs() * mean(err_g * n.abs()) + 20 * H * spread), n

        d, err, out_gain = ds, torch.zeros_like(ds), (None, None)
        if gain is not None:
            q = (offset + gain) * dy
            part, err, n = through(s, q, 2 * H * q.abs())
            d = ds + part
            err = err + H * d.abs()
            out_gain = total(dy * n, 7 * H * (dy * n).abs(), dgain)
        dh = out_post = out_gate = (None, None)
        if h is not None:
            w = torch.ones(1, self.D, dtype=torch.float64) if gate is None else gate_rows(gate, T)
            v = scale * w * d
            err_v = (scale * w).abs() * err + 2 * H * v.abs()
            if post is not None:
                g = (offset + post) * v
                dh_, err_h, m = through(h, g, (offset + post).abs() * err_v + 2 * H * g.abs())
                out_post = total(v * m, m.abs() * err_v + 9 * H * (v * m).abs(), dpost)
                u = (offset + post) * m
            else:
                dh_, err_h, u = v, err_v, h
            dh = dh_, err_h
            if gate is not None:
                rows = gate.view(-1, self.D).shape[0]
                terms, te = scale * d * u, (scale * u).abs() * err + 12 * H * (scale * d * u).abs()
                out_gate = total(terms.view(rows, T // rows, self.D), te.view(rows, T // rows, self.D),
                                 dgate.view(rows, self.D) if dgate is not None else None)
        return (d, err), dh, out_gain, out_post, out_gate


SIZES = [(1, 1), (1, 16), (2, 4096), (3, 7), (5, 255), (2, 257), (9, 1024), (7, 1025), (300, 100), (33, 2048), (3, 4097),
         (2, 16384), (4, 16383), (700, 515), (1, 8192), (130, 2050)]


def forms(T):
    """(post, gate rows, block, gain, pad, shift, scale, offset)."""
    some = next((g for g in (7, 5, 3, 2) if T % g == 0), 1)
    return [(True, 1, True, True, 0, 0, 1.0, 0.0), (True, 0, True, True, 8, 0, 0.25, 1.0),
            (False, 0, True, True, 0, 1, 1.0, 0.0), (True, some, True, True, 3, 1, 0.7, 0.0),
            (True, T, True, False, 0, 0, 1.0, 1.0), (False, some, True, True, 0, 0, -1.5, 0.0),
            (False, T, True, True, 1, 0, 1.0, 0.0), (False, 0, False, True, 8, 0, 1.0, 1.0),
            (False, 1, True, False, 0, 0, 0.5, 0.0)]


@pytest.mark.parametrize("kind", DT)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_forward(size, kind):
    T, D = size
    gen = torch.Generator().manual_seed(T * 31 + D)
    step = half_step(kind)
    for post, gate, block, gain, pad, shift, scale, offset in forms(T):
        c = Case(gen, T, D, kind, post, gate, block, gain, pad, shift, scale, offset)
        s, y = norm.forward(c.x, c.gain, **c.kw())
        want_s, err_s, want_y, err_y = c.forward64()
        if block:
            inside("s", s, want_s, err_s + step * (want_s.abs() + err_s))
        else:
            assert s is c.x
        if gain:
            inside("y", y, want_y, err_y + step * (want_y.abs() + err_y))
        else:
            assert y is None
        # into given outputs: between their rows nothing changes; in place too
        hold = torch.full((2, T, D + pad), 7.0, dtype=DT[kind], device="cuda")
        s2, y2 = norm.forward(c.x, c.gain, out=hold[0, :, :D] if block else None,
                              out_norm=hold[1, :, :D] if gain else None, **c.kw())
        assert torch.equal(s2, s) and (not gain or torch.equal(y2, y)) and bool((hold[:, :, D:] == 7).all())
        if block:
            for at in ("x", "h"):
                work = dict(x=c.x.clone(), h=c.h.clone())
                kw = {**c.kw(), "h": work["h"]}
                s2, y2 = norm.forward(work["x"], c.gain, out=work[at], **kw)
                assert s2.data_ptr() == work[at].data_ptr() and torch.equal(s2, s)
                assert not gain or torch.equal(y2, y)
        if gain:
            work = c.x.clone()
            assert torch.equal(norm.forward(work, c.gain, out_norm=work, **c.kw())[1], y)


def check_backward(c, s, grad, keep, given):
    g = DT[grad]
    gen = torch.Generator().manual_seed(3)
    olds = [None if p is None else randn(gen, tuple(p.shape), grad) for p in (c.gain, c.post, c.gate)]
    bufs = [None if o is None else o.clone() for o in olds] if given else [None] * 3
    out = norm.backward(c.dy, s, c.gain, ds=c.ds, dgain=bufs[0], dpost_gain=bufs[1], dgate=bufs[2], accumulate=keep,
                        grad_dtype=g, **c.kw())
    want = c.backward64(s, *olds, keep)
    for name, got, (v, err), k in zip(("dx", "dh", "dgain", "dpost_gain", "dgate"), out, want,
                                      [c.kind] * 2 + [grad] * 3):
        if v is None:
            assert got is None, name
            continue
        inside(name, got.view(v.shape), v, err + half_step(k) * (v.abs() + err))
    for b, o in zip(bufs, out[2:]):
        assert b is None or b.data_ptr() == o.data_ptr()
    return out


@pytest.mark.parametrize("kind, grad", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_backward(size, kind, grad):
    T, D = size
    gen = torch.Generator().manual_seed(T * 17 + D)
    for k, (post, gate, block, gain, pad, shift, scale, offset) in enumerate(forms(T)):
        c = Case(gen, T, D, kind, post, gate, block, gain, pad, shift, scale, offset)
        s = randn(gen, (T, D), kind, 2.0, pad=pad, shift=shift)
        out = check_backward(c, s, grad, k % 2 == 0, True)
        new = norm.backward(c.dy, s, c.gain, ds=c.ds, grad_dtype=DT[grad], **c.kw())
        assert all(a is None or torch.equal(a, b) for a, b in zip(new[:2], out[:2]))
        if k % 2:
            assert all(a is None or torch.equal(a, b) for a, b in zip(new[2:], out[2:]))
        few = norm.backward(c.dy, s, c.gain, ds=c.ds, need_params=False, **c.kw())
        assert few[2:] == (None, None, None) and torch.equal(few[0], out[0])
        only = norm.backward(c.dy, s, c.gain, ds=c.ds, need_dx=False, need_dh=False, grad_dtype=DT[grad], **c.kw())
        assert only[:2] == (None, None)
        assert all(a is None or torch.equal(a, b) for a, b in zip(only[2:], new[2:]))


@pytest.mark.parametrize("size", [(40000, 24, 5), (40000, 24, 2), (40000, 24, 20000), (40000, 24, 1), (5000, 300, 4),
                                  (1400, 4100, 7), (1400, 4100, 4), (6000, 1100, 100), (6000, 1100, 3000)], ids=str)
@pytest.mark.parametrize("kind, grad", [("bf16", "bf16"), ("f32", "f32")])
def test_gate_rows_over_runs(size, kind, grad):
    """Gate rows of several tokens each, ending anywhere in a workgroup's runs."""
    T, D, per = size
    gen = torch.Generator().manual_seed(T + D + per)
    for post, keep in ((True, False), (False, True)):
        c = Case(gen, T, D, kind, post, T // per, True, True, scale=0.5)
        check_backward(c, randn(gen, (T, D), kind, 2.0), grad, keep, True)


def test_without_tokens():
    for kind in DT:
        x, w = torch.zeros(0, 40, dtype=DT[kind], device="cuda"), torch.ones(40, dtype=DT[kind], device="cuda")
        gates = torch.ones(3, 40, dtype=DT[kind], device="cuda")
        s, y = norm.forward(x, w, h=x, post_gain=w, gate=gates)
        assert s.shape == y.shape == (0, 40)
        for gate in (w, gates):
            for keep in (False, True):
                bufs = [torch.full(v.shape, 3.0, device="cuda") for v in (w, w, gate)]
                norm.backward(x, x, w, h=x, post_gain=w, gate=gate, dgain=bufs[0], dpost_gain=bufs[1], dgate=bufs[2],
                              accumulate=keep)
                assert all(bool((b == (3.0 if keep else 0.0)).all()) for b in bufs)


def test_without_a_later_gradient():
    gen = torch.Generator().manual_seed(4)
    c = Case(gen, 20, 300, "f32", True, 1, True, True)
    c.ds = torch.zeros_like(c.ds)
    s = randn(gen, (20, 300), "f32")
    a = norm.backward(c.dy, s, c.gain, **c.kw())
    b = norm.backward(c.dy, s, c.gain, ds=c.ds, **c.kw())
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_values_of_any_size():
    """Squares past fp32's range either way, zero rows, and rows of NaN and
    infinity, which stay in their rows."""
    gen = torch.Generator().manual_seed(5)
    base = randn(gen, (6, 100), "f32")
    w, wp = randn(gen, (100,), "f32", 0.1, 1.0), randn(gen, (100,), "f32", 0.1, 1.0)
    size = torch.tensor([1e30, 1e-30, 1e19, 1.0, 1e37, 1e-37], device="cuda")[:, None]
    x = base * size
    _, y = norm.forward(x, w, eps=0.0)
    n = host(x) / mean(host(x) ** 2).sqrt()
    want = n * host(w)
    inside("y", y, want, 10 * H * want.abs())
    s, y = norm.forward(torch.zeros_like(x), w, h=x, post_gain=wp, eps=0.0)
    want = n * host(wp)
    inside("s", s, want, 10 * H * want.abs())
    dy = randn(gen, (6, 100), "f32")
    dx, _, dgain, _, _ = norm.backward(dy, x, w, eps=0.0)
    q = host(dy) * host(w)
    want = (q - n * mean(q * n)) / mean(host(x) ** 2).sqrt()
    bound = 20 * H * (q.abs() + n.abs() * mean((q * n).abs())) / mean(host(x) ** 2).sqrt() + 2.0 ** -148
    rows = [0, 2, 3, 4, 1]                     # the last row's gradient passes fp32's range
    inside("dx", dx[rows], want[rows], bound[rows])
    terms = host(dy) * n
    inside("dgain", dgain, terms.sum(0), 60 * H * terms.abs().sum(0))
    for kind in DT:
        for D in (40, 300, 3000, 9000):
            x, h = randn(gen, (5, D), kind), randn(gen, (5, D), kind)
            g, p = randn(gen, (D,), kind), randn(gen, (D,), kind)
            x[0], h[0] = 0, 0
            s, y = norm.forward(x, g, h=h, post_gain=p)
            assert not s[0].any() and not y[0].any()
            bad = h.clone()
            bad[1, 3], bad[2, D - 1] = float("nan"), float("inf")
            s2, y2 = norm.forward(x, g, h=bad, post_gain=p)
            assert bool(y2[1].isnan().all()) and bool(y2[2].isnan().all())
            assert torch.equal(s2[[0, 3, 4]], s[[0, 3, 4]]) and torch.equal(y2[[0, 3, 4]], y[[0, 3, 4]])
            clean, dirty = (norm.backward(x, s, g, h=v, post_gain=p) for v in (h, bad))
            for a, b in zip(clean[:2], dirty[:2]):
                assert torch.equal(a[[0, 3, 4]], b[[0, 3, 4]])
            assert torch.equal(clean[2], dirty[2]) and bool(dirty[3].isnan().all())


def test_gradients_match_differences():
    """Central differences of the definition in 64 bits, step 1e-4: off by 1e-8 of
    third derivatives and 1e-12 of rounding, beside the fp32 gradients' 2^-18 of
    the sums' size."""
    gen = torch.Generator().manual_seed(6)
    T, D, gates, scale, offset = 6, 11, 2, 0.6, 1.0
    x, h = randn(gen, (T, D), "f32"), randn(gen, (T, D), "f32")
    gain, post, gate = randn(gen, (D,), "f32", 0.3), randn(gen, (D,), "f32", 0.3), randn(gen, (gates, D), "f32")
    dy, ds = randn(gen, (T, D), "f32"), randn(gen, (T, D), "f32")

    def loss(x, h, gain, post, gate):
        u = (offset + post) * h / (mean(h * h) + 1e-6).sqrt()
        s = x + scale * gate.repeat_interleave(T // gates, 0) * u
        y = (offset + gain) * s / (mean(s * s) + 1e-6).sqrt()
        return (host(dy) * y).sum() + (host(ds) * s).sum()

    s, _ = norm.forward(x, gain, h=h, post_gain=post, gate=gate, scale=scale, offset=offset)
    dx, dh, dgain, dpost, dgate = norm.backward(dy, s, gain, ds=ds, h=h, post_gain=post, gate=gate, scale=scale,
                                                offset=offset)
    args = [host(v) for v in (x, h, gain, post, gate)]
    for at, got in enumerate((dx, dh, dgain, dpost, dgate)):
        base = args[at]
        for i in range(0, base.numel(), 3):
            e = torch.zeros(base.numel(), dtype=torch.float64)
            e[i] = 1e-4
            e = e.view(base.shape)
            up, down = list(args), list(args)
            up[at], down[at] = base + e, base - e
            d = (loss(*up) - loss(*down)) / 2e-4
            tol = (1e-6 + 2.0 ** -18) * host(dy).abs().sum()
            assert abs(host(got).view(-1)[i] - d) < tol


def test_in_place_and_shapes():
    gen = torch.Generator().manual_seed(7)
    c = Case(gen, 24, 130, "bf16", True, 4, True, True)
    want_s, want_y = norm.forward(c.x, c.gain, **c.kw())
    kw = {**c.kw(), "h": c.h.view(2, 3, 4, 130)}
    s, y = norm.forward(c.x.view(2, 3, 4, 130), c.gain, **kw)
    assert s.shape == y.shape == (2, 3, 4, 130)
    assert torch.equal(s.view(24, 130), want_s) and torch.equal(y.view(24, 130), want_y)
    back = norm.backward(c.dy.view(2, 3, 4, 130), s, c.gain, ds=c.ds.view(2, 3, 4, 130), **kw)
    flat = norm.backward(c.dy, want_s, c.gain, ds=c.ds, **c.kw())
    assert all(torch.equal(a.reshape(b.shape), b) for a, b in zip(back, flat))
    # a row's outputs over its inputs, through the library's own entry point
    for over_x, over_h in (("ds", "dy"), ("dy", "h"), ("s", "h"), ("h", "ds")):
        w = dict(dy=c.dy.clone(), ds=c.ds.clone(), s=want_s.clone(), h=c.h.clone())
        n = dc.dc_norm_backward_workspace(0, 24, 130, 4)
        ws = torch.empty(n, dtype=torch.uint8, device="cuda")
        dc.dc_norm_backward(0, 24, 130, w["dy"], 130, w["ds"], 130, w["s"], 130, w["h"], 130, c.post, c.gate, 4, 130,
                            c.gain, 1.0, 0.0, c.eps, w[over_x], 130, w[over_h], 130, 1, None, None, None, 0, 0, ws, n)
        assert torch.equal(w[over_x], flat[0]) and torch.equal(w[over_h], flat[1])


@pytest.mark.parametrize("D", [40, 600, 4096, 9001])
def test_outputs_over_both_inputs(D):
    """s over x with y over h, and the other way round."""
    gen = torch.Generator().manual_seed(12)
    c = Case(gen, 19, D, "bf16", True, 1, True, True)
    want = norm.forward(c.x, c.gain, **c.kw())
    for s_over, y_over in (("x", "h"), ("h", "x")):
        w = dict(x=c.x.clone(), h=c.h.clone())
        got = norm.forward(w["x"], c.gain, out=w[s_over], out_norm=w[y_over], **{**c.kw(), "h": w["h"]})
        assert got[0] is w[s_over] and got[1] is w[y_over]
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_rows_too_long_are_refused():
    x, w = torch.zeros(2, 16385, device="cuda"), torch.zeros(16385, device="cuda")
    with pytest.raises(dc.DCError) as e:
        norm.forward(x, w)
    assert e.value.code == dc.DC_ERR_UNSUPPORTED
    red = deferred.DeferredReducer(1, 20000)
    red.acc.fill_(7.0)
    with pytest.raises(dc.DCError):
        red.accumulate_norm(0, x, x, w, gain_at=0)
    assert bool((red.acc == 7).all()) and not red.open


def test_offsets_past_32_bits():
    gen = torch.Generator().manual_seed(8)
    big = torch.zeros(33 * (1 << 26), dtype=torch.bfloat16, device="cuda").view(33, 1 << 26)
    far, near = [], []
    for k in range(5):
        far.append(big[:, 200 * k + 3:200 * k + 93])
        near.append(randn(gen, (33, 90), "bf16"))
        far[-1].copy_(near[-1])
    g, p = randn(gen, (90,), "bf16"), randn(gen, (90,), "bf16")
    want = norm.forward(near[0], g, h=near[1], post_gain=p, gate=near[4])
    got = norm.forward(far[0], g, h=far[1], post_gain=p, gate=far[4], out=big[:, 2000:2090], out_norm=big[:, 3001:3091])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    want = norm.backward(near[2], near[0], g, ds=near[3], h=near[1], post_gain=p, gate=near[4], grad_dtype=torch.bfloat16)
    got = norm.backward(far[2], far[0], g, ds=far[3], h=far[1], post_gain=p, gate=far[4], dgate=big[:, 4001:4091],
                        grad_dtype=torch.bfloat16)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    T = (1 << 21) + 5
    x = torch.ones(T, 1030, dtype=torch.bfloat16, device="cuda")
    w = torch.full((1030,), 2.0, dtype=torch.bfloat16, device="cuda")
    _, y = norm.forward(x, w, eps=0.0)
    assert bool((y[0] == 2).all()) and bool((y[-1] == 2).all()) and bool((y[T // 2] == 2).all())
    dx, _, dgain, _, _ = norm.backward(x, x, w, ds=x, eps=0.0)
    assert bool((dx[0] == 1).all()) and bool((dx[-1] == 1).all()) and bool((dgain - T).abs().max() <= (T + 40) * H * T)


def both(c):
    s, y = norm.forward(c.x, c.gain, **c.kw())
    return [s, y] + list(norm.backward(c.dy, s, c.gain, ds=c.ds, **c.kw()))


@pytest.mark.parametrize("size", [(3, 4096, 1), (500, 513, 5), (60, 9000, 60)], ids=str)
def test_replayed_and_on_other_streams(size):
    T, D, gates = size
    gen = torch.Generator().manual_seed(9)
    sets = [Case(gen, T, D, "bf16", True, gates, True, True) for _ in range(3)]
    want = [both(c) for c in sets]
    torch.cuda.synchronize()
    names = ("x", "h", "post", "gain", "gate", "dy", "ds")
    static = Case(gen, T, D, "bf16", True, gates, True, True)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        rec = both(static)
    for c, w in list(zip(sets, want)) * 2:
        for n in names:
            getattr(static, n).copy_(getattr(c, n))
        graph.replay()
        both(sets[1])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(rec, w))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = []
    for rep in range(4):
        c, st = sets[rep % 2], streams[rep % 2]
        s, y = norm.forward(c.x, c.gain, stream=st, **c.kw())
        got.append([s, y] + list(norm.backward(c.dy, s, c.gain, ds=c.ds, stream=st.cuda_stream, **c.kw())))
    torch.cuda.synchronize()
    for rep, g in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(g, want[rep % 2]))


def test_into_the_deferred_reduction():
    """Gains and gates of two replicas over two micro-batches: the accumulators
    hold what the same calls give in buffers of their own."""
    W, T, D = 2, 30, 50
    gen = torch.Generator().manual_seed(10)
    red = deferred.DeferredReducer(W, 400)
    for step in range(2):
        red.acc.fill_(float("nan"))
        bufs = [[torch.zeros(D, device="cuda"), torch.zeros(D, device="cuda"), torch.zeros(3, D, device="cuda")]
                for _ in range(W)]
        for mb in range(2):
            for r in range(W):
                c = Case(gen, T, D, "bf16", True, 3, True, True)
                s, _ = norm.forward(c.x, c.gain, **c.kw())
                b = bufs[r]
                want = norm.backward(c.dy, s, c.gain, ds=c.ds, dgain=b[0], dpost_gain=b[1], dgate=b[2], accumulate=True,
                                     **c.kw())
                got = red.accumulate_norm(r, c.dy, s, c.gain, ds=c.ds, gain_at=3, post_gain_at=60, gate_at=117, **c.kw())
                assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
            red.end_micro_batch()
        out = torch.zeros(1, red.ld, device="cuda")
        red.reduce(out, red.ld)
        for at, k in ((3, 0), (60, 1), (117, 2)):
            for r in range(W):
                assert torch.equal(red.acc[r, at:at + bufs[r][k].numel()], bufs[r][k].view(-1))
        assert not out[0, 53:60].any() and not out[0, 110:117].any() and not out[0, 267:400].any()
    c = Case(gen, T, D, "bf16", True, 3, True, True)
    over = dict(dy=c.dy, s=c.x, gain=c.gain, ds=c.ds, gain_at=3, post_gain_at=60, gate_at=117, **c.kw())
    for bad in (dict(gain_at=351), dict(gate_at=-1), dict(gate_at=100), dict(row=2), dict(dy=c.dy[:4]),
                dict(gain=None, dy=None), dict(scale=float("inf"))):
        before = red.acc.clone()
        with pytest.raises(ValueError):
            red.accumulate_norm(**{**dict(row=0), **over, **bad})
        assert torch.equal(red.acc, before) and not red.open


@pytest.mark.parametrize("D", [40, 300, 4096, 4097, 9000])
def test_without_a_norm_after_the_block_its_output_does_not_matter(D):
    """dh = scale gate dx where h is not normed: infinities and NaN in h (of
    tokens that a gate of zeros shuts out) leave it alone."""
    gen = torch.Generator().manual_seed(D)
    for kind in DT:
        ds, h, gate = randn(gen, (6, D), kind), randn(gen, (6, D), kind), randn(gen, (3, D), kind)
        h[1, 3], h[2, D - 1], h[3] = float("nan"), float("inf"), float("-inf")
        gate[1] = 0
        for g in (None, gate[0], gate):
            dx, dh, *_ = norm.backward(None, ds, ds=ds, h=h, gate=g, scale=0.5, need_params=False)
            assert torch.equal(dx, ds)
            want = host(ds) * 0.5 * (1.0 if g is None else gate_rows(host(g), 6))
            inside("dh", dh, want, (half_step(kind) + 2 * H) * want.abs())


@pytest.mark.parametrize("D", [40, 300, 2500, 6000, 9001])
@pytest.mark.parametrize("kind", DT)
def test_subnormal_rows(kind, D):
    """With eps = 0 a row of subnormal values has a factor 1 / rms past fp32's
    range, and values of order 1 all the same.  Bounds as above; a gradient
    through such a row is rounded to fp32 or bf16 once more."""
    gen = torch.Generator().manual_seed(D)
    T, step = 5, half_step(kind)
    unit = randn(gen, (T, D), "f32", 1.0)
    sizes = torch.tensor([1.0, 3e-40, 2e-39, 1e-39 if kind == "bf16" else 4e-42, 1e-38], dtype=torch.float64)
    tiny = (unit.double() * sizes.cuda()[:, None]).to(DT[kind])
    tiny[:, D // 2] = 0
    w, wp = randn(gen, (D,), kind, 0.1, 1.0), randn(gen, (D,), kind, 0.1, 1.0)
    v = host(tiny)
    rms = mean(v * v).sqrt()
    n = v / rms
    _, y = norm.forward(tiny, w, eps=0.0)
    want = n * host(w)
    inside("y", y, want, 12 * H * want.abs() + step * want.abs() * 1.01)
    s, y = norm.forward(torch.zeros_like(tiny), w, h=tiny, post_gain=wp, eps=0.0)
    want = n * host(wp)
    inside("s", s, want, 12 * H * want.abs() + step * want.abs() * 1.01)
    # every gradient so small that 1 / rms times it stays in range
    dy, gates = randn(gen, (T, D), kind, 2.0 ** -30), randn(gen, (T, D), kind)
    dx, _, dgain, _, _ = norm.backward(dy, tiny, w, eps=0.0)

    def through(g):
        return (g - n * mean(g * n)) / rms, 24 * H * (g.abs() + n.abs() * mean((g * n).abs())) / rms

    want, err = through(host(dy) * host(w))
    inside("dx", dx, want, err + step * (want.abs() + err))
    terms = host(dy) * n
    inside("dgain", dgain, terms.sum(0), 60 * H * terms.abs().sum(0))
    ds = randn(gen, (T, D), kind, 2.0 ** -30)
    for gate in (None, gates):
        dx, dh, _, dpost, dgate = norm.backward(None, ds, ds=ds, h=tiny, post_gain=wp, gate=gate, eps=0.0)
        assert torch.equal(dx, ds)
        v = host(ds) * (1.0 if gate is None else host(gate))
        want, err = through(v * host(wp))
        inside("dh", dh, want, err + step * (want.abs() + err))
        terms = v * n
        inside("dpost", dpost, terms.sum(0), 60 * H * terms.abs().sum(0))
        if gate is not None:
            want = host(ds) * n * host(wp)
            inside("dgate", dgate, want, 20 * H * want.abs())


@pytest.mark.parametrize("size", [(16384, 64, 2), (16384, 64, 12), (4000, 74, 8), (4000, 300, 2), (9000, 1100, 3)],
                         ids=str)
@pytest.mark.parametrize("kind", DT)
def test_gate_sums_do_not_drift(size, kind):
    """Sums of many equal terms, whose roundings all fall to one side.  A part is
    one run's: a fused add and a product's rounding for each of its few rows.
    Parts are added in 64 bits, so that the bound does not grow with their
    number: (2 run + 4) 2^-24 of the sum, and half a step of bf16's own values
    nowhere, as these are exact.  Runs are as in the library: one workgroup of
    512 threads a compute unit, 16, 64 or 256 threads to a row."""
    T, D, gates = size
    T = T // gates * gates
    gen = torch.Generator().manual_seed(D)
    ds = (0.3 + torch.rand(1, D, generator=gen)).to(DT[kind]).expand(T, D).contiguous().cuda()
    h = (0.7 + torch.rand(1, D, generator=gen)).to(DT[kind]).expand(T, D).contiguous().cuda()
    gate = torch.ones(gates, D, dtype=DT[kind], device="cuda")
    dgate = norm.backward(None, ds, ds=ds, h=h, gate=gate)[4]
    n = 16 if kind == "bf16" else 8
    threads = 16 if D <= 16 * n else 64 if D <= 64 * n else 256
    run = -(-T // (256 * 512 // threads))
    want = (host(ds) * host(h))[:1] * (T // gates)
    inside("dgate", dgate, want.expand(gates, D), (2 * run + 4) * H * want.abs())

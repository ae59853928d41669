"""Orthogonalising and the matrix update on the GPU against their definition
in 64 bits.

The bound on |error|_F is carried through the steps.  With u the half step of
what X, A and B are held in (one fp16 2^-11, a pair of them 2^-22) and
g(k) = 2 k 2^-23 for a sum of k products:
  dA <= u |A| + g(n) |X|^2
  dB <= (|b| + 2 |c| |A|_2) dA + u |B| + g(m) |c| |A|^2 + 2^-21 (|b| |A| + |c| |A|^2)
  injected in X <= u |X'| + |X|_2 dB + g(m) |B| |X| + 2^-21 (|a| |X| + |B| |X|)
and an error that is there grows by at most the largest slope of the step's
polynomial over the singular values' range (the map is odd and acts on
singular values).  A tenth is added for products of errors.  The output is
rounded by finfo.eps / 2."""
import numpy as np
import pytest

from gradient_reduction_amd import dc, executor, muon
from synth import workloads as wl

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


def half_step(dtype):
    return T().finfo(dtype).eps / 2


def reference(u, steps, coeffs, eps, kind, u_err=0.0):
    """(O in 64 bits, bound on the error's Frobenius norm before the output's
    rounding) for one matrix U known to u_err |U|_F."""
    t = T()
    hold = 2.0 ** -11 if kind == "bf16" else 2.0 ** -22
    flip = u.shape[0] > u.shape[1]
    x = u.t() if flip else u
    x = x / (x.norm() + eps)
    m, n = x.shape
    err = (hold + 2.0 ** -21 + 2 * u_err) * x.norm().item() + (m * n) ** 0.5 * 2.0 ** -34
    top = 1.0
    for a, b, c in coeffs:
        f = lambda z: z.norm().item()                                    # noqa: E731
        two = lambda z: t.linalg.matrix_norm(z, 2).item()                # noqa: E731
        ab, cb, aa = abs(float(b)), abs(float(c)), abs(float(a))
        A = x @ x.t()
        B = float(b) * A + float(c) * (A @ A)
        new = float(a) * x + B @ x
        dA = hold * f(A) + 2 * n * STEP * f(x) ** 2
        dB = ((ab + 2 * cb * two(A)) * dA + hold * f(B) + 2 * m * STEP * cb * f(A) ** 2
              + 2.0 ** -21 * (ab * f(A) + cb * f(A) ** 2))
        dX = hold * f(new) + two(x) * dB + 2 * m * STEP * f(B) * f(x) + 2.0 ** -21 * (aa * f(x) + f(B) * f(x))
        top = max(top, two(x)) + err
        s = np.linspace(0, top, 2000)
        slope = np.abs(float(a) + 3 * float(b) * s ** 2 + 5 * float(c) * s ** 4).max()
        err = slope * err + dX
        x = new
    return (x.t() if flip else x), 1.1 * err


def check(name, got, u, kind, steps=5, coeffs=None, eps=1e-7, out_eps=None, u_err=0.0):
    t = T()
    co = np.tile(np.array(muon.COEFFS, np.float32), (steps, 1)) if coeffs is None else np.asarray(coeffs, np.float32)
    want, bound = reference(u, steps, co, eps, kind, u_err)
    got = got.cpu().double()
    assert bool(t.isfinite(got).all()), f"{name}: not finite"
    off = (got - want).norm().item()
    bound += (out_eps if out_eps is not None else 0.0) * (want.norm().item() + bound)
    assert off <= bound, f"{name}: off by {off:.3g}, bound {bound:.3g}, |O| {want.norm().item():.3g}"


def gradient(gen, *shape, dtype, strong=3):
    t = T()
    g = t.randn(*shape, generator=gen, dtype=t.float64)
    u = t.randn(*shape[:-1], strong, generator=gen, dtype=t.float64)
    v = t.randn(*shape[:-2], strong, shape[-1], generator=gen, dtype=t.float64)
    return ((g + 0.3 * u @ v) * 1e-3).to(dtype).cuda()


SHAPES = [(1, 1), (1, 2), (2, 1), (1, 333), (333, 1), (3, 5), (5, 3), (8, 8), (16, 64), (63, 65), (64, 64), (65, 64),
          (129, 127), (128, 128), (130, 300), (300, 130), (257, 513), (200, 1000)]


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_one_list_of_every_shape(kind):
    t = T()
    gen = t.Generator().manual_seed(1)
    gs = [gradient(gen, r, c, dtype=dt(kind)) for r, c in SHAPES]
    outs = muon.orthogonalize(gs)
    for (r, c), g, o in zip(SHAPES, gs, outs):
        assert o.shape == g.shape and o.dtype == g.dtype
        check(f"{r} x {c}", o, g.cpu().double(), kind, out_eps=half_step(dt(kind)))
        alone = muon.orthogonalize(g)         # a list's other members change nothing but the tile size
        check(f"{r} x {c} alone", alone, g.cpu().double(), kind, out_eps=half_step(dt(kind)))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(60, 3, 17, 24), (300, 24, 40), (2, 512, 640), (5, 640, 512)], ids=str)
def test_batches(shape, kind):
    """More matrices than one launch takes, and enough tiles for the large
    tile."""
    t = T()
    gen = t.Generator().manual_seed(2)
    g = gradient(gen, *shape, dtype=dt(kind))
    o = muon.orthogonalize(g)
    flat_g, flat_o = g.reshape(-1, *shape[-2:]), o.reshape(-1, *shape[-2:])
    for k in list(range(0, len(flat_g), max(1, len(flat_g) // 6))) + [len(flat_g) - 1]:
        check(f"{k}", flat_o[k], flat_g[k].cpu().double(), kind, out_eps=half_step(dt(kind)))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_large_tiles_with_odd_sizes(kind):
    t = T()
    gen = t.Generator().manual_seed(4)
    gs = [gradient(gen, 1100, 2090, dtype=dt(kind)), gradient(gen, 3001, 515, dtype=dt(kind)),
          gradient(gen, 7, 11, dtype=dt(kind))]
    for hold in ("auto", "one", "pair"):
        held = {"auto": kind, "one": "bf16", "pair": "f32"}[hold]
        for g, o in zip(gs, muon.orthogonalize(gs, hold=hold)):
            check(f"{tuple(g.shape)} {hold}", o, g.cpu().double(), held, out_eps=half_step(dt(kind)))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_strides_places_and_in_place(kind):
    """Gradients at odd places with row strides, outputs interleaved as
    columns of one buffer whose other columns stay, and results over their own
    gradients: the same values as contiguous ones."""
    t = T()
    gen = t.Generator().manual_seed(3)
    h = dt(kind)
    for r, c in [(70, 50), (50, 70), (130, 131)]:
        g = gradient(gen, 2, r, c, dtype=h)
        want = muon.orthogonalize(g)
        buf = t.full((2, r, c + 5), float("nan"), dtype=h, device="cuda").view(-1)
        odd = t.full((buf.numel() + 1,), float("nan"), dtype=h, device="cuda")[1:].view(2, r, c + 5)[:, :, :c]
        odd.copy_(g)
        assert t.equal(muon.orthogonalize(odd), want)
        both = t.full((r, 2 * c + 3), 7.0, dtype=h, device="cuda")
        muon.orthogonalize([odd[0], odd[1]], out=[both[:, :c], both[:, c + 2:2 * c + 2]])
        assert t.equal(both[:, :c], want[0]) and t.equal(both[:, c + 2:2 * c + 2], want[1])
        assert bool((both[:, c:c + 2] == 7).all()) and bool((both[:, 2 * c + 2:] == 7).all())
        same = g.clone()
        assert t.equal(muon.orthogonalize(same, out=same), want) and t.equal(same, want)


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_zero_and_bad_matrices(kind):
    """A zero matrix gives zero; NaN and infinity stay in their matrix;
    sizes at the ends of the type's range are normalised."""
    t = T()
    gen = t.Generator().manual_seed(5)
    h = dt(kind)
    g = gradient(gen, 6, 40, 90, dtype=h)
    clean = muon.orthogonalize(g)
    bad = g.clone()
    bad[0] = 0
    bad[1, 3, 4] = float("nan")
    bad[2, 39, 89] = float("inf")
    bad[4] *= 2.0 ** 100
    bad[5] *= 2.0 ** 30
    o = muon.orthogonalize(bad)
    assert bool((o[0] == 0).all()) and bool(t.isnan(o[1]).all()) and bool(t.isnan(o[2]).all())
    assert t.equal(o[3], clean[3])
    for k in (4, 5):
        check(f"scaled {k}", o[k], bad[k].cpu().double(), kind, out_eps=half_step(h))
    tiny = (g[3].double() * 2.0 ** -90).to(h)      # |G| far under eps: scaled by 1 / eps
    check("tiny", muon.orthogonalize(tiny, eps=1e-30), tiny.cpu().double(), kind, eps=float(np.float32(1e-30)),
          out_eps=half_step(h))
    assert bool(t.isnan(muon.orthogonalize(t.zeros(3, 4, dtype=h, device="cuda"), eps=0.0)).all())
    assert muon.orthogonalize([]) == [] and muon.orthogonalize(t.zeros(0, 3, 4, dtype=h, device="cuda")).numel() == 0


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("coeffs", [
    [(1.5, -0.5, 0.0)], [(1.5, -0.5, 0.0)] * 16, [(15 / 8, -10 / 8, 3 / 8)] * 4,
    [(8.28, -23.59, 17.3), (4.1, -2.95, 0.55), (1.875, -1.25, 0.375)], [(0.0, 0.0, 0.0)], [(2.0, 0.0, 0.0)] * 5,
], ids=["cubic", "cubic16", "quintic", "by-step", "zero", "linear"])
def test_other_steps(coeffs, kind):
    t = T()
    gen = t.Generator().manual_seed(6)
    g = gradient(gen, 90, 70, dtype=dt(kind))
    o = muon.orthogonalize(g, steps=len(coeffs), coeffs=coeffs)
    check("steps", o, g.cpu().double(), kind, steps=len(coeffs), coeffs=coeffs, out_eps=half_step(dt(kind)))


@pytest.mark.parametrize("kind, wkind", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("nesterov, scale", [(True, "rms"), (False, "aspect"), (True, "none")])
@pytest.mark.parametrize("choice", ["auto", "one"])
def test_update(kind, wkind, nesterov, scale, choice):
    t = T()
    gen = t.Generator().manual_seed(7)
    shapes = [(1, 1), (3, 40), (40, 3), (65, 130), (200, 120), (2, 66, 67)]
    gs = [gradient(gen, *s, dtype=dt(kind)) for s in shapes]
    ms = [(t.randn(*s, generator=gen) * 1e-3).cuda() for s in shapes]
    hold = [t.full(s[:-1] + (s[-1] + 3,), 7.0, dtype=dt(wkind), device="cuda") for s in shapes]
    ws = [h[..., :-3] for h in hold]
    for w in ws:
        w.copy_((t.randn(w.shape, generator=gen) * 0.05).to(dt(wkind)))
    lr, mu, wd = np.float32(0.02), np.float32(0.95), np.float32(0.1)
    lrs = t.tensor([0.5], device="cuda")
    for step, scalar in ((0, None), (1, lrs)):
        w0, m0 = [w.cpu().double() for w in ws], [m.cpu().double() for m in ms]
        muon.update(ws, gs, ms, lr=float(lr), mu=float(mu), nesterov=nesterov, weight_decay=float(wd), scale=scale,
                    hold=choice, lr_scale=scalar)
        rate = float(lr) * (0.5 if scalar is not None else 1.0)
        for k, s in enumerate(shapes):
            rows, cols = s[-2:]
            f = {"none": 1.0, "aspect": max(1.0, rows / cols) ** 0.5, "rms": 0.2 * max(rows, cols) ** 0.5}[scale]
            g = gs[k].cpu().double()
            m = float(mu) * m0[k] + g
            assert bool(((ms[k].cpu().double() - m).abs() <= 2.0 ** -24 * m.abs() + 1e-40).all())
            u = float(mu) * m + g if nesterov else m
            got, old = ws[k].cpu().double(), w0[k]
            flat = [v.reshape(-1, rows, cols) for v in (u, got, old, g, m)]
            for uu, ww, oo, gg, mm in zip(*flat):
                # u: two fused multiply-adds, each off by half a step of its result
                du = (2.0 ** -24 * (mm.norm() + uu.norm()) / uu.norm()).item()
                held = "bf16" if choice == "one" or (kind == wkind == "bf16" and min(rows, cols) >= 256) else "f32"
                o, bound = reference(uu, 5, np.tile(np.array(muon.COEFFS, np.float32), (5, 1)), 1e-7, held, du)
                want = oo * (1 - rate * float(wd)) - rate * f * o
                bound = (rate * f * bound + 6 * 2.0 ** -24 * (oo.norm() + rate * f * o.norm()).item()
                         + half_step(dt(wkind)) * want.norm().item()) * 1.01
                assert (ww - want).norm().item() <= bound, (s, step, (ww - want).norm().item(), bound)
    assert all(bool((h[..., -3:] == 7).all()) for h in hold)


def test_replayed_and_on_other_streams():
    """A recorded update follows a learning rate in device memory; replays
    with eager work between, and two lists at once on two streams, give the
    eager results bit for bit."""
    t = T()
    gen = t.Generator().manual_seed(8)
    shapes = [(64, 96), (300, 200), (1, 7)]
    gs = [gradient(gen, *s, dtype=t.bfloat16) for s in shapes]
    w0 = [(t.randn(*s, generator=gen) * 0.05).cuda() for s in shapes]

    def fresh():
        return [w.clone() for w in w0], [t.zeros_like(w) for w in w0]

    rates = [1.0, 0.5, 0.25, 0.0]
    we, me = fresh()
    want = []
    for r in rates:
        muon.update(we, gs, me, lr=0.02, lr_scale=t.tensor([r], device="cuda"))
        want.append([w.clone() for w in we])
    wr, mr = fresh()
    rate = t.ones(1, device="cuda")
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        muon.update(wr, gs, mr, lr=0.02, lr_scale=rate)
    for r, ww in zip(rates, want):
        rate.fill_(r)
        g.replay()
        muon.orthogonalize(gs)                # eager work with a workspace of its own
        t.cuda.synchronize()
        for a, b in zip(wr, ww):
            assert t.equal(a, b)
    eager = muon.orthogonalize(gs)
    streams = [t.cuda.Stream() for _ in range(2)]
    outs = []
    for rep in range(3):
        for st in streams:
            st.wait_stream(t.cuda.current_stream())
            outs.append(muon.orthogonalize(gs, stream=st))
    t.cuda.synchronize()
    for o in outs:
        for a, b in zip(o, eager):
            assert t.equal(a, b)


def test_offsets_past_32_bits():
    t = T()
    ld = (1 << 25) + 24
    big = t.empty(70 * ld, dtype=t.bfloat16, device="cuda")
    far = big.view(70, ld)[:, 5:105]
    gen = t.Generator().manual_seed(9)
    g = gradient(gen, 70, 100, dtype=t.bfloat16)
    far.copy_(g)
    want = muon.orthogonalize(g)
    assert t.equal(muon.orthogonalize(far), want)
    assert t.equal(muon.orthogonalize(g, out=big.view(70, ld)[:, 200:300]), want)


@pytest.mark.parametrize("dtype", [wl.DT_BF16, wl.DT_F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("owners", [True, False], ids=["owner", "allreduce"])
def test_flush_then_owners_update(owners, dtype):
    """The whole step: rank slabs flushed to their owners (or to every rank),
    then the matrix parameters' update from the flushed slab, against the
    update of the flushed gradients taken out by hand."""
    t = T()
    sizes = [(40, 30), None, (64, 64), (7, 200), None, (200, 7), (129, 65)]
    numel = [a[0] * a[1] if a else 77 for a in sizes]
    w = wl.custom_flush("update", 4, dtype, numel, capacity=9000, pre_div=1, value_seed=3)
    eb = t.bfloat16 if dtype == wl.DT_BF16 else t.float32
    gen = t.Generator().manual_seed(12)
    slab = (t.randn(w.W, w.ld, generator=gen) * 1e-3).to(eb).cuda()
    out = t.zeros_like(slab)
    ex = executor.from_workload(w, reduce_to_owner=owners)
    ex.build_owner_map()
    ex.plan()
    weights = {p: (t.randn(*s, generator=gen) * 0.05).cuda() for p, s in enumerate(sizes) if s}
    momenta = {p: t.zeros_like(v) for p, v in weights.items()}
    ex.register_matrices(weights, momenta)
    co = np.tile(np.array(muon.COEFFS, np.float32), (5, 1))
    lr, mu, wd = float(np.float32(0.02)), float(np.float32(0.95)), float(np.float32(0.1))
    for step in range(2):
        old = {p: (weights[p].cpu().double(), momenta[p].cpu().double()) for p in weights}
        for b in range(len(w.buckets)):
            ex.flush(b, slab, w.ld, out, w.ld)
        ex.muon_update(out, w.ld, lr=0.02, weight_decay=0.1)
        t.cuda.synchronize()
        for bk in w.buckets:
            for task in bk.tasks:
                p = task.param
                if not sizes[p]:
                    continue
                row = max(int(ex.h_owner[p]) if owners else -1, 0)
                c0 = bk.col + task.offset
                g = out[row, c0:c0 + numel[p]].cpu().double()
                mean = slab[:, c0:c0 + numel[p]].cpu().double().mean(0)
                assert (g - mean).norm() <= 0.02 * mean.norm()      # it is the flushed gradient
                g = g.view(*sizes[p])
                m = mu * old[p][1] + g
                assert bool(((momenta[p].cpu().double() - m).abs() <= 2.0 ** -24 * m.abs() + 1e-40).all())
                u = mu * m + g
                du = (2.0 ** -24 * (m.norm() + u.norm()) / u.norm()).item()
                o, bound = reference(u, 5, co, 1e-7, "f32", du)     # fp32 weights: pairs
                f = lr * 0.2 * max(sizes[p]) ** 0.5
                want = old[p][0] * (1 - lr * wd) - f * o
                bound = (f * bound + 7 * 2.0 ** -24 * (want.norm() + f * o.norm()).item()) * 1.01
                assert (weights[p].cpu().double() - want).norm().item() <= bound
    z2 = executor.from_workload(w, reduce_to_owner=False, zero2=True)
    with pytest.raises(ValueError):
        z2.register_matrices(weights, momenta)
    with pytest.raises(ValueError):
        ex.register_matrices({1: t.zeros(7, 12, device="cuda")}, {1: t.zeros(7, 12, device="cuda")})
    with pytest.raises(ValueError):
        ex.register_matrices(weights, {})


def test_owners_update_refusals():
    """Refused on the host: an update of nothing, a slab that does not hold
    every matrix, a rate that is not one element."""
    t = T()
    w = wl.custom_flush("update", 2, wl.DT_F32, [12 * 8, 77], capacity=9000, pre_div=1, value_seed=3)
    slab = t.zeros(w.W, w.ld, device="cuda")
    ex = executor.from_workload(w, reduce_to_owner=True)
    ex.build_owner_map()
    with pytest.raises(RuntimeError):
        ex.muon_update(slab, w.ld, lr=0.02)
    weights, momenta = {0: t.ones(12, 8, device="cuda")}, {0: t.ones(12, 8, device="cuda")}
    ex.register_matrices(weights, momenta)
    for bad in (slab.bfloat16(), slab.cpu(), slab[:, :50].contiguous()[:1]):
        with pytest.raises(ValueError):
            ex.muon_update(bad, w.ld, lr=0.02)
    for rate in (t.ones(2, device="cuda"), t.ones(1), t.ones(1, device="cuda").double()):
        with pytest.raises(ValueError):
            ex.muon_update(slab, w.ld, lr=0.02, lr_scale=rate)
        with pytest.raises(ValueError):
            muon.update(weights[0], slab[0, :96].view(12, 8), momenta[0], lr=0.02, lr_scale=rate)
    assert bool((weights[0] == 1).all()) and bool((momenta[0] == 1).all())

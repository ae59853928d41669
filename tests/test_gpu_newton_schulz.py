"""Orthogonalised matrices and updates on the GPU, held to the bounds of
newton_schulz_model (which zeros, -O, a step less or a lost low half break:
tests/test_newton_schulz_bounds.py)."""
import pytest
import torch

from gradient_reduction_amd import dc, executor, muon
from synth import workloads as wl
from tests import newton_schulz_model as ns
from tests import product_forms as pf

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    dc.lib()
    yield
    torch.cuda.synchronize()


def dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def close(name, got, u, hold, coeffs=ns.COEFFS, eps=1e-7):
    got = got.cpu()
    assert bool(torch.isfinite(got).all()), f"{name}: not finite"
    off = ns.beyond(got, ns.exact(u, coeffs, eps).cpu(), torch.finfo(got.dtype).eps / 2)
    most = 1.01 * ns.bound(hold, tuple(u.shape))
    assert off <= most, f"{name}: off by {off:.3g} |O| beyond the output's rounding, bound {most:.3g}"


@pytest.mark.parametrize("shape", [(768, 130), (1024, 1024)], ids=str)
def test_halves_are_of_one_number(shape):
    """Ten matrices held in pairs: a low half that belongs to another rounding
    than the stored high half shows in some of them."""
    us = torch.stack([ns.gradient(torch.Generator().manual_seed(s), *shape, dtype=torch.float32)
                      for s in range(10)])
    got = muon.orthogonalize(us.cuda(), hold="pair")
    off = [ns.beyond(g, ns.exact(u, ns.COEFFS, 1e-7), 2.0 ** -24) for g, u in zip(got.cpu(), us)]
    print("beyond the output's rounding, |O|:", " ".join(f"{v:.2g}" for v in off), flush=True)
    assert max(off) <= 1.01 * ns.PAIR_BOUND


@pytest.mark.parametrize("shape", [(300, 260), (257, 1025), (1024, 1024)], ids=str)
def test_fewer_bits_are_the_callers_choice(shape):
    """A caller who says nothing gets pairs: on bf16 matrices too, nothing is
    lost beyond the output's own rounding."""
    u = ns.gradient(torch.Generator().manual_seed(3), *shape, dtype=torch.bfloat16)
    close("orthogonalize", muon.orthogonalize(u.cuda()), u, "pair")
    close("one", muon.orthogonalize(u.cuda(), hold="one"), u, "one")
    w = torch.zeros(*shape, dtype=torch.bfloat16, device="cuda")
    m = torch.zeros(*shape, device="cuda")
    # from zero weights and momenta, w = -O
    muon.update(w, u.cuda(), m, lr=1.0, mu=0.0, nesterov=False, scale="none")
    close("update", -w, u, "pair")


def test_update_after_a_refused_registration():
    """The executor's update after a registration that was refused steps the
    matrices that were registered before, from their own gradients."""
    sizes = [(40, 30), (64, 64), (7, 200)]
    w = wl.custom_flush("update", 4, wl.DT_F32, [a * b for a, b in sizes], capacity=9000, pre_div=1, value_seed=3)
    gen = torch.Generator().manual_seed(12)
    slab = (torch.randn(w.W, w.ld, generator=gen) * 1e-3).cuda()
    out = torch.zeros_like(slab)
    ex = executor.from_workload(w, reduce_to_owner=True)
    ex.build_owner_map()
    weights = {p: torch.zeros(*s, device="cuda") for p, s in enumerate(sizes)}
    ex.register_matrices(weights, {p: torch.zeros_like(v) for p, v in weights.items()})
    with pytest.raises(ValueError):
        ex.register_matrices({0: torch.zeros(40, 31, device="cuda")}, {0: torch.zeros(40, 31, device="cuda")})
    for b in range(len(w.buckets)):
        ex.flush(b, slab, w.ld, out, w.ld)
    ex.muon_update(out, w.ld, lr=1.0, mu=0.0, nesterov=False, scale="none")
    for bk in w.buckets:
        for t in bk.tasks:
            u = slab[:, bk.col + t.offset:bk.col + t.offset + t.numel].cpu().double().mean(0)
            # the flushed fp32 sum of four rows is off by 3 roundings of 2^-24 at
            # most, which the steps' slopes (10 on the average) make 2e-6
            want = ns.exact(u.view(*sizes[t.param]), ns.COEFFS, 1e-7)
            assert ns.error(-weights[t.param].cpu().double(), want) <= ns.PAIR_BOUND + 2e-6 + 2.0 ** -24


@pytest.mark.parametrize("hold", ["one", "pair"])
def test_a_list_of_more_than_one_workspace(hold):
    """Matrices whose planes do not fit the workspace together: those at the
    beginning, the end and the middle, the first of a new chunk among them."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    us = [(torch.randn(*s, generator=gen, device="cuda") * 1e-3).bfloat16()
          for s in [(4096, 4096)] * 9 + [(600, 270), (5000, 4100), (4096, 4096), (4096, 11008)] + [(4096, 4096)] * 24]
    got = muon.orthogonalize(us, hold=hold)
    # 16 of the pairs fit 4 GiB, 32 held once
    for k in (0, 8, 9, 10, 12, 15, 16, 17, 31, 32, 36):
        close(k, got[k], us[k], hold)


def made(shapes, dtype, seed):
    gen = torch.Generator().manual_seed(seed)
    some = [ns.gradient(gen, *s, dtype=dtype) for s in sorted(set(shapes))]
    # matrices of one shape differ by a shift of their columns
    return [some[sorted(set(shapes)).index(s)].roll(k, 1).cuda().contiguous() for k, s in enumerate(shapes)]


@pytest.mark.parametrize("hold", ["one", "pair"])
@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("shapes", pf.ORTHOGONAL, ids=lambda v: f"{len(v)}x{v[0]}".replace(" ", ""))
def test_every_form_of_the_products(shapes, kind, hold):
    us = made(shapes, dt(kind), 5)
    got = muon.orthogonalize(us, hold=hold)
    for k in {0, len(shapes) // 2, len(shapes) - 1}:
        close(k, got[k], us[k], hold)


@pytest.mark.parametrize("hold", ["one", "pair"])
@pytest.mark.parametrize("kind, wkind", [("bf16", "f32"), ("bf16", "bf16"), ("f32", "f32")])
@pytest.mark.parametrize("shapes", pf.ORTHOGONAL, ids=lambda v: f"{len(v)}x{v[0]}".replace(" ", ""))
def test_every_form_of_the_update(shapes, kind, wkind, hold):
    """w <- (1 - lr wd) w - lr O(mu m + g).  The look-ahead is rounded twice to
    fp32 (2^-24 of it each), which the steps make ten times as much on the
    average; the weight takes six roundings of its terms besides the output's."""
    gs = made(shapes, dt(kind), 6)
    gen = torch.Generator(device="cuda").manual_seed(7)
    ms = [torch.randn(*s, generator=gen, device="cuda") * 1e-3 for s in shapes]
    ws = [(torch.randn(*s, generator=gen, device="cuda") * 0.05).to(dt(wkind)) for s in shapes]
    some = sorted({0, len(shapes) // 2, len(shapes) - 1})
    old = {k: (ws[k].double(), ms[k].double()) for k in some}
    lr, mu, wd = 0.5, 0.9375, 0.125                     # exact in fp32
    muon.update(ws, gs, ms, lr=lr, mu=mu, nesterov=True, weight_decay=wd, scale="none", hold=hold)
    for k in some:
        w, m = old[k]
        new = mu * m + gs[k].double()
        assert bool(((ms[k].double() - new).abs() <= 2.0 ** -24 * new.abs() + 1e-40).all())
        o = lr * ns.exact(mu * new + gs[k].double(), ns.COEFFS, 1e-7)
        want = (1 - lr * wd) * w - o
        half = torch.finfo(ws[k].dtype).eps / 2
        off = (ws[k].double() - want).abs() - half * want.abs() - 6 * 2.0 ** -24 * (w.abs() + o.abs())
        most = 1.02 * (ns.bound(hold, shapes[k]) + 20 * 2.0 ** -24)
        assert (off.clamp(min=0).norm() / o.norm()).item() <= most, k


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("shape", [(1, 1), (1, 2), (2, 1), (1, 333), (333, 1), (3, 5), (5, 3), (8, 8), (16, 64), (63, 65),
                                   (64, 64), (65, 64), (129, 127), (300, 130), (257, 513), (200, 1000)], ids=str)
def test_every_shape(shape, kind):
    u = ns.gradient(torch.Generator().manual_seed(8), *shape, dtype=dt(kind))
    close("pair", muon.orthogonalize(u.cuda()), u, "pair")
    close("one", muon.orthogonalize(u.cuda(), hold="one"), u, "one")
    close("four steps", muon.orthogonalize(u.cuda(), steps=4), u, "pair", coeffs=ns.COEFFS[:4])
    # another gradient's size, and eps that counts beside it
    v = (u.double() * 1e4).to(u.dtype)
    close("large", muon.orthogonalize(v.cuda()), v, "pair")
    eps = float(torch.tensor(u.double().norm().item() / 4).float())
    close("eps", muon.orthogonalize(u.cuda(), eps=eps), u, "pair", eps=eps)


@pytest.mark.parametrize("shape", [(20, 2000), (4000, 24), (48, 4096)], ids=str)
def test_long_sums(shape):
    """Sums of thousands of products are added up in parts of 256 (32 times
    eight): off by what the model of that gives.  One matrix's error scatters by
    a third about it, the mean of eight by an eighth; twice that is allowed.
    Sums in one piece are off by 1.6, 2 and 1.15 times as much."""
    us = [ns.gradient(torch.Generator().manual_seed(s), *shape, dtype=torch.float32) for s in range(8)]
    got = muon.orthogonalize(torch.stack(us).cuda(), hold="pair").cpu()
    here = there = 0.0
    for g, u in zip(got, us):
        want = ns.exact(u, ns.COEFFS, 1e-7)
        here += ns.error(g.double(), want) / len(us)
        there += ns.error(ns.model(u, ns.COEFFS, 1e-7, "pair", fold=32), want) / len(us)
    print(f"{shape}: {here:.3g}, the model {there:.3g}", flush=True)
    assert here <= 1.25 * there


@pytest.mark.parametrize("shape", [(1, 300), (300, 1), (4, 1000), (8, 300)], ids=str)
def test_few_rows_keep_every_product(shape):
    """With few singular values roundings do not average, and the product of the
    low halves, 2^-24 of a value and of one sign on A's diagonal, counts.  The
    mean of 64 matrices, which scatter by a half about the model's, is within an
    eighth of it; without that product 1.2 to 1.6 times as much is left."""
    us = [ns.gradient(torch.Generator().manual_seed(s), *shape, dtype=torch.float32) for s in range(64)]
    got = muon.orthogonalize(torch.stack(us).cuda(), hold="pair").cpu()
    here = there = other = 0.0
    for g, u in zip(got, us):
        want = ns.exact(u, ns.COEFFS, 1e-7)
        here += ns.error(g.double(), want) / len(us)
        there += ns.error(ns.model(u, ns.COEFFS, 1e-7, "pair", fold=32, lows=True), want) / len(us)
        other += ns.error(ns.model(u, ns.COEFFS, 1e-7, "pair", fold=32), want) / len(us)
    print(f"{shape}: {here:.3g}, the model {there:.3g}, without the product {other:.3g}", flush=True)
    assert here <= 1.125 * there + 2.0 ** -25         # and the output's own rounding

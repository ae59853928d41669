"""A whole step as a user runs it: an embedding that is the output's matrix
too, a block between two norms with a gate, two replicas of two micro-batches
into the deferred reduction, clipping by the global norm and the owner's
update; against the same model differentiated by torch in 64 bits.

Bound.  The operators' own tests hold each to its roundings; here fp32 runs
through a dozen of them one behind the other, each off by a few 2^-22 of its
operands' sizes, over sums of up to 200 terms: 2^-14 of the largest gradient
(and of a clipped one) is over 100 such steps in a row.  The update is held to 4e-6 of its
orthogonalised matrix (the pairs' error), which the gradient's error joins."""
import numpy as np
import pytest
import torch

from gradient_reduction_amd import clip, dc, deferred, embedding, linear, muon, norm

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    dc.lib()
    yield
    torch.cuda.synchronize()


V, D, F, B, S = 50, 40, 72, 4, 9       # B sequences of S tokens, a gate row each
SHAPES = {"table": (V, D), "pre": (D,), "up": (F, D), "up_b": (F,), "down": (D, F), "post": (D,), "gate": (B, D),
          "last": (D,)}
AT, M = {}, 0
for _name, _shape in SHAPES.items():
    AT[_name] = M
    M += int(np.prod(_shape))
SCALE, DEPTH = D ** 0.5, 0.5


def model64(p, ids, dlogits):
    """The loss whose gradients the step adds up."""
    def rms(v, g):
        return (1 + g) * v / (v.square().mean(-1, keepdim=True) + 1e-6).sqrt()

    ok = (ids >= 0)[..., None]
    x = torch.where(ok, p["table"][ids.clamp(min=0)] * SCALE, 0.0).view(B * S, D)
    h = torch.nn.functional.gelu(rms(x, p["pre"]) @ p["up"].t() + p["up_b"]) @ p["down"].t()
    s = x + DEPTH * p["gate"].repeat_interleave(S, 0) * rms(h, p["post"])
    return (dlogits * (rms(s, p["last"]) @ p["table"].t())).sum()


def layers(red, row, p, ids, dlogits):
    """Forward and backward of one micro-batch of one replica."""
    x = embedding.forward(ids, p["table"], scale=SCALE).view(B * S, D)
    _, n = norm.forward(x, p["pre"], offset=1.0)
    a, pre = linear.forward(n, p["up"], p["up_b"], act="gelu", save_pre=True)
    h = linear.forward(a, p["down"])
    around = dict(h=h, post_gain=p["post"], gate=p["gate"], scale=DEPTH, offset=1.0)
    s, y = norm.forward(x, p["last"], **around)
    linear.forward(y, p["table"])
    dy = red.accumulate_linear(row, AT["table"], dlogits, y, p["table"])
    dx, dh = red.accumulate_norm(row, dy, s, p["last"], gain_at=AT["last"], post_gain_at=AT["post"], gate_at=AT["gate"],
                                 **around)
    da = red.accumulate_linear(row, AT["down"], dh, a, p["down"])
    dn = red.accumulate_linear(row, AT["up"], da, n, p["up"], pre, "gelu", bias_offset=AT["up_b"])
    dx, _ = red.accumulate_norm(row, dn, x, p["pre"], ds=dx, offset=1.0, gain_at=AT["pre"])
    red.accumulate_embedding(row, AT["table"], dx.view(B, S, D), ids, V, scale=SCALE)


@pytest.mark.parametrize("max_norm", [0.5, 1e9])
def test_step(max_norm):
    gen = torch.Generator().manual_seed(1)
    W, micro = 2, 2
    p = {k: (torch.randn(s, generator=gen) * (s[-1] ** -0.5 if len(s) > 1 else 0.2)).cuda() for k, s in SHAPES.items()}
    red = deferred.DeferredReducer(W, M)
    out = torch.zeros(1, red.ld, device="cuda")
    momenta = {k: torch.zeros(SHAPES[k], device="cuda") for k in ("up", "down")}
    for step in range(2):
        p64 = {k: v.cpu().double().requires_grad_() for k, v in p.items()}
        loss = 0.0
        for _ in range(micro):
            for r in range(W):
                ids = torch.randint(-1, V, (B, S), generator=gen)
                dlogits = torch.randn(B * S, V, generator=gen) * 0.1
                loss = loss + model64(p64, ids, dlogits.double())
                layers(red, r, p, ids.cuda(), dlogits.cuda())
            red.end_micro_batch()
        red.reduce(out, red.ld)
        want = dict(zip(SHAPES, torch.autograd.grad(loss, [p64[k] for k in SHAPES])))
        for k, g in want.items():
            got = out[0, AT[k]:AT[k] + g.numel()].view(g.shape).cpu().double()
            assert (got - g).abs().max() <= 2.0 ** -14 * g.abs().max(), k
        total = sum((g ** 2).sum() for g in want.values()).sqrt().item()
        n = red.clip(out, red.ld, max_norm)
        assert abs(n.item() - total) <= 2.0 ** -14 * total
        c = min(1.0, max_norm / (total + 1e-6))
        grads = {k: out[0, AT[k]:AT[k] + g.numel()].view(g.shape) for k, g in want.items()}
        for k, g in want.items():
            assert (grads[k].cpu().double() - c * g).abs().max() <= 2.0 ** -13 * c * g.abs().max(), k
        names = ("up", "down")
        before = {k: p[k].clone() for k in names}
        kept = {k: momenta[k].clone() for k in names}
        muon.update([p[k] for k in names], [grads[k] for k in names], [momenta[k] for k in names], lr=0.02)
        for k in names:
            m = 0.95 * kept[k].double() + grads[k].double()
            assert (momenta[k].double() - m).abs().max() <= 2.0 ** -22 * m.abs().max()
            assert bool(torch.isfinite(p[k]).all()) and not torch.equal(p[k], before[k])
        for k in SHAPES:
            if k not in names:
                p[k] -= 0.02 * grads[k]


def test_step_as_a_graph():
    """Forward, backward, reduction and clipping recorded once and replayed on
    other tokens, with eager work between."""
    gen = torch.Generator().manual_seed(2)
    p = {k: (torch.randn(s, generator=gen) * (s[-1] ** -0.5 if len(s) > 1 else 0.2)).cuda() for k, s in SHAPES.items()}
    red = deferred.DeferredReducer(1, M)
    sets = [(torch.randint(-1, V, (B, S), generator=gen).cuda(), torch.randn(B * S, V, generator=gen).cuda())
            for _ in range(3)]

    def step(red, ids, dlogits, out):
        layers(red, 0, p, ids, dlogits)
        red.end_micro_batch()
        red.reduce(out, red.ld)
        return red.clip(out, red.ld, 0.5)

    eager = []
    for s in sets:
        out = torch.zeros(1, red.ld, device="cuda")
        eager.append((step(red, *s, out), out))
    torch.cuda.synchronize()
    static, out = [v.clone() for v in sets[0]], torch.zeros(1, red.ld, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm_ = step(red, *static, out)
    other, spare = deferred.DeferredReducer(1, M), torch.zeros(1, red.ld, device="cuda")
    for s, (n, o) in list(zip(sets, eager)) * 2:
        for a, b in zip(static, s):
            a.copy_(b)
        graph.replay()
        step(other, *sets[1], spare)
        torch.cuda.synchronize()
        assert torch.equal(norm_, n) and torch.equal(out, o)


def test_clipping_a_list_between_reduction_and_update():
    """The owner's matrices clipped as a list, their update scale-free: an
    orthogonalised step is the same with and without clipping."""
    gen = torch.Generator().manual_seed(3)
    gs = [torch.randn(s, generator=gen).cuda() for s in ((64, 48), (40, 130), (33, 33))]
    want = muon.orthogonalize([g.clone() for g in gs])
    n = clip.clip_grad_norm(gs, 0.125)
    assert abs(clip.grad_norm(gs).item() - 0.125) <= 1e-6 and n.item() > 10
    for a, b in zip(muon.orthogonalize(gs), want):
        # both within 4e-6 of the exact one; eps = 1e-7 against norms of 0.05 moves it by 2e-6 (slope under 20 of tiny values)
        assert (a - b).norm() <= 5e-5 * b.norm()

"""The bounds that the GPU's orthogonalised matrices are held to can fail: the
kernels' roundings stay under half of them, and wrong outputs do not (on the
CPU; see newton_schulz_model)."""
import numpy as np
import pytest
import torch

from gradient_reduction_amd import dc
from tests import newton_schulz_model as ns

SHAPES = [(1, 1), (1, 333), (333, 1), (3, 5), (8, 8), (16, 64), (63, 65), (128, 128), (300, 130), (257, 513),
          (512, 640)]


def made(shape, seed):
    gen = torch.Generator().manual_seed(seed)
    return ns.gradient(gen, *shape, dtype=torch.bfloat16)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_bounds_separate(shape):
    for seed in range(3):
        u = made(shape, seed)
        want = ns.exact(u, ns.COEFFS, 1e-7)
        for hold in ("pair", "one"):
            most = ns.bound(hold, shape)
            assert ns.error(ns.model(u, ns.COEFFS, 1e-7, hold), want) <= most / 2
            for wrong in (torch.zeros_like(want), -want, ns.exact(u, ns.COEFFS[:4], 1e-7),
                          ns.exact(u, ns.COEFFS[:3], 1e-7)):
                assert ns.error(wrong, want) > most
                for out in (torch.bfloat16, torch.float32):
                    half = torch.finfo(out).eps / 2
                    assert ns.beyond(wrong.to(out), want, half) > 1.01 * most
        half = torch.finfo(torch.float32).eps / 2
        dropped = ns.model(u, ns.COEFFS, 1e-7, "pair", "no low half")
        assert ns.beyond(dropped.float(), want, half) > 1.01 * ns.PAIR_BOUND
        if min(shape) >= 63:      # also behind a bf16 output's rounding
            half = torch.finfo(torch.bfloat16).eps / 2
            assert ns.beyond(dropped.bfloat16(), want, half) > 1.01 * ns.PAIR_BOUND


@pytest.mark.parametrize("shape", [(768, 130), (1024, 1024)], ids=str)
def test_halves_of_two_roundings_are_seen(shape):
    """A low half that is not the stored high half's breaks the bound on some of
    ten seeds; halves of one number never come near it."""
    worst = 0.0
    for seed in range(10):
        u = made(shape, seed)
        want = ns.exact(u, ns.COEFFS, 1e-7)
        worst = max(worst, ns.error(ns.model(u, ns.COEFFS, 1e-7, "pair", "folded"), want))
        if seed < 2:
            assert ns.error(ns.model(u, ns.COEFFS, 1e-7, "pair"), want) <= ns.PAIR_BOUND / 2
    assert worst > ns.PAIR_BOUND


def layer_7b():
    return [(4096, 4096)] * 4 + [(11008, 4096)] * 2 + [(4096, 11008)]


@pytest.mark.parametrize("hold", [dc.DC_HOLD_ONE, dc.DC_HOLD_PAIR])
def test_the_workspace_does_not_grow_with_the_model(hold):
    """A list's matrices share one workspace of a few GiB (or of the largest
    matrix), however many there are."""
    def need(shapes):
        m = np.zeros(len(shapes), dc.MATRIX_DTYPE)
        m["rows"], m["cols"] = [s[0] for s in shapes], [s[1] for s in shapes]
        return dc.dc_orthogonalize_workspace(dc.DC_BF16, dc.DC_F32, hold, m, len(m))

    parts = 1 << 20
    for shapes in (layer_7b() * 32, [(8192, 8192)] * 100, [(1 << 20, 512)] * 9, layer_7b()[::-1] * 5):
        assert need(shapes) <= max((4 << 30) + parts, max(need([s]) for s in set(shapes)))
    # what fits is not cut: one layer, and 128 small matrices
    one = 2 * hold * 2
    assert need(layer_7b()) >= one * sum(a * b + min(a, b) ** 2 for a, b in layer_7b())
    assert need([(1024, 1024)] * 128) >= one * 128 * 2 * 1024 * 1024

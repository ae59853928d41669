"""The Newton-Schulz steps in 64 bits, and a model of how the kernels round
them: what the bounds on an orthogonalised matrix are taken from.

The bounds are on |error|_F / |O|_F before the output's own rounding.  A value
held as a pair of fp16 is off by at most 2^-23 of itself (the high half leaves
at most 2^-11 of the value, of which the low half keeps 11 bits and a sign), a
product of pairs leaves out low x low (2^-24), and sums round to 24 bits: about
2^-22 of a value in all, once in each of A, B and X per step.  A rounding in X
grows by the slopes of the steps that follow: 3.45^5 = 485 where all five meet a
vanishing singular value, about ten on the average over a random matrix's.
model() carries exactly these roundings through and, with sums rounded once, gives 4e-7 to 6e-7 at sides
of 16 and more, up to 2e-6 on a few elements, and 1.2e-3 to 1.8e-3 (up to 4.5e-3)
with one fp16.  The bounds are twice the largest of these;
tests/test_newton_schulz_bounds.py checks that, and that wrong outputs break
them.
"""
import numpy as np
import torch

COEFFS = np.tile(np.array([3.4445, -4.7750, 2.0315], np.float32), (5, 1))
PAIR_BOUND = 4e-6
ONE_BOUND = 4e-3          # smaller side of 256 and more
ONE_BOUND_SMALL = 1e-2    # under it: few singular values average less


def bound(hold, shape):
    """Of |error|_F / |O|_F, before the output's rounding."""
    if hold == "pair":
        return PAIR_BOUND
    return ONE_BOUND if min(shape[-2:]) >= 256 else ONE_BOUND_SMALL


def gradient(gen, *shape, dtype, strong=3):
    """Noise and a few strong directions, as a batch's weight gradient has."""
    g = torch.randn(*shape, generator=gen, dtype=torch.float64)
    u = torch.randn(*shape[:-1], strong, generator=gen, dtype=torch.float64)
    v = torch.randn(*shape[:-2], strong, shape[-1], generator=gen, dtype=torch.float64)
    return ((g + 0.3 * torch.matmul(u, v)) * 1e-3).to(dtype)


def exact(u, coeffs, eps):
    """O of one matrix [rows, cols] in 64 bits."""
    u = u.double()
    x = u.t() if u.shape[0] > u.shape[1] else u
    x = x / (x.norm() + eps)
    for a, b, c in coeffs:
        g = x @ x.t()
        x = float(a) * x + (float(b) * g + float(c) * (g @ g)) @ x
    return x.t().contiguous() if u.shape[0] > u.shape[1] else x


def _held(v, hold, fault):
    """(high, low) halves of fp32 values v; unrounded: what a conversion that
    is folded into a multiplication rounds instead."""
    v32 = v.float()
    high = v32.half()
    # (numpy rounds 64 bits to 16 once; torch does it by way of 32)
    sub = torch.from_numpy(v.numpy().astype(np.float16)) if fault == "folded" else high
    low = (v32 - sub.float()).half() if hold == "pair" else torch.zeros_like(high)
    if fault == "no low half":
        low = torch.zeros_like(high)
    return high.double(), low.double()


def _instructions(a, b, acc, fold):
    """acc + a b as the matrix instructions add it up: eight products at a time,
    each cut off at 2^-24 of the largest one's power of two, and their sum
    rounded into the fp32 sum; after `fold` of these a sum begins anew, and the
    sums are added up apart (0: never)."""
    part = torch.zeros_like(acc) if fold else acc
    for i, k in enumerate(range(0, a.shape[1], 8)):
        p = a[:, k:k + 8, None] * b[None, k:k + 8, :]
        unit = torch.exp2(torch.floor(torch.log2(p.abs().amax(1, keepdim=True).clamp(min=1e-300))) - 24)
        part = (part + (torch.trunc(p / unit) * unit).sum(1)).float().double()
        if fold and (i + 1) % fold == 0:
            acc, part = (acc + part).float().double(), torch.zeros_like(acc)
    return (acc + part).float().double() if fold else part


def _product(a, b, fold=None, lows=False):
    """Of (high, low) pairs, summed in fp32: rounded once, or with `fold` as the
    instructions do it (the small products first); low x low with `lows`."""
    if fold is None:
        return (a[0] @ b[0] + a[0] @ b[1] + a[1] @ b[0]).float().double()
    acc = torch.zeros(a[0].shape[0], b[0].shape[1], dtype=torch.float64)
    if lows:
        acc = _instructions(a[1], b[1], acc, 0)
    acc = _instructions(a[0], b[1], _instructions(a[1], b[0], acc, 0), 0)
    return _instructions(a[0], b[0], acc, fold)


def model(u, coeffs, eps, hold, fault=None, fold=None, lows=False):
    """O as the kernels round it (before the output's rounding).  fold, lows:
    products as _product gives them.  fault: "no low half", or "folded" (the low half taken from another rounding of
    the value than the one that is stored, in B)."""
    x = u.double()
    flip = u.shape[0] > u.shape[1]
    x = x.t() if flip else x
    scale = 2.0 ** 13
    own = None if fault == "folded" else fault
    p = _held((x * (scale / (x.norm() + eps))).float().double(), hold, own)
    for k, (a, b, c) in enumerate(coeffs):
        a, b, c = float(a), float(b), float(c)
        # A by a power of two
        g = _held((_product(p, (p[0].t(), p[1].t()), fold, lows) * (2.0 ** 12 / scale ** 2)), hold, own)
        # B = alpha (beta A + A A), alpha no power of two
        alpha = torch.tensor(c * 2.0 ** 11 / 2.0 ** 24).float().double()
        beta = torch.tensor(b * 2.0 ** 12 / c).float().double()
        s = (_product(g, g, fold, lows) + beta * (g[0] + g[1])).float().double()
        q = _held((alpha * s).contiguous(), hold, fault)
        new = (a * 2.0 ** 11 * (p[0] + p[1]) + _product(q, p, fold, lows)).float().double() * 2.0 ** -11
        if k + 1 < len(coeffs):
            p = _held(new, hold, own)
    out = new / scale
    return out.t().contiguous() if flip else out


def error(got, want):
    return ((got - want).norm() / want.norm()).item()


def beyond(got, want, step):
    """|what got is off by beyond the half step of its type|_F / |want|_F: a
    value that is rounded from want + e is off by at most e + step (|want| +
    |e|), so this is at most (1 + step) |e|_F / |want|_F."""
    off = (got.double() - want).abs() - step * want.abs()
    return (off.clamp(min=0).norm() / want.norm()).item()

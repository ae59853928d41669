"""Orthogonalised updates of whole matrices on torch tensors.

After reduce-to-owner one rank holds a parameter's whole reduced gradient
(DeepSpeed issue "[REQUEST] DeepCompile ZeRO-1: reduce-to-owner instead of
AllReduce", problem statement), which is what orthogonalising a matrix needs:
update() takes the momentum's step, orthogonalises it by Newton-Schulz
products and steps the weights; orthogonalize() is the middle part alone.

A tensor [..., rows, cols] is a batch of matrices; one call takes a list of
tensors of any shapes.  Marshalling only: everything runs in libdc.so
(dc_orthogonalize, dc_muon_update) on `stream`, or on torch's current stream
of the tensors' device; workspaces come from torch's allocator.  Nothing here
is seen by autograd.
"""
import numpy as np
import torch

from . import dc
from .linear import dtype_of, on, workspace

# The quintic a s + b s^3 + c s^5 whose slope at 0 lifts small singular values
# fastest while five steps bring all of them near 1.
COEFFS = (3.4445, -4.7750, 2.0315)
HOLDS = {"auto": dc.DC_HOLD_AUTO, "one": dc.DC_HOLD_ONE, "pair": dc.DC_HOLD_PAIR}
SCALES = {"none": dc.DC_SCALE_NONE, "aspect": dc.DC_SCALE_ASPECT, "rms": dc.DC_SCALE_RMS}


def _steps(steps, coeffs):
    """[steps, 3] from one triple or one per step."""
    c = np.asarray(coeffs, np.float32)
    if c.shape == (3,):
        return np.ascontiguousarray(np.broadcast_to(c, (steps, 3)))
    if c.shape != (steps, 3):
        raise ValueError(f"coeffs of shape {c.shape}, expected (3,) or ({steps}, 3)")
    return np.ascontiguousarray(c)


def _addresses(name, t):
    """(addresses of a batch's matrices, row stride in elements)."""
    if t.dim() < 2:
        raise ValueError(f"{name} of shape {tuple(t.shape)} is no matrix")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: columns must be contiguous (strides {t.stride()})")
    a = np.array([t.data_ptr()], np.uint64)
    for d in range(t.dim() - 2):
        step = np.arange(t.shape[d], dtype=np.uint64) * np.uint64(t.stride(d) * t.element_size())
        a = (a[:, None] + step).ravel()
    return a, t.stride(-2) if t.shape[-2] > 1 else t.shape[-1]


def matrices(grads, outs, momenta=None):
    """MATRIX_DTYPE records of lists of tensors of the same shapes."""
    recs = []
    for k, (g, o) in enumerate(zip(grads, outs)):
        m = momenta[k] if momenta is not None else None
        for name, t in (("out", o), ("momentum", m)):
            if t is not None and t.shape != g.shape:
                raise ValueError(f"{name} {k} of shape {tuple(t.shape)}, its gradient's is {tuple(g.shape)}")
        ga, ld_g = _addresses(f"gradient {k}", g)
        if g.numel() == 0:
            continue
        r = np.zeros(len(ga), dc.MATRIX_DTYPE)
        r["grad"], r["ld_grad"] = ga, ld_g
        r["out"], r["ld_out"] = _addresses(f"out {k}", o)
        if m is not None:
            r["momentum"], ld_m = _addresses(f"momentum {k}", m)
            if ld_m != g.shape[-1]:
                raise ValueError(f"momentum {k}: rows must be contiguous (strides {m.stride()})")
        r["rows"], r["cols"] = g.shape[-2], g.shape[-1]
        recs.append(r)
    return np.concatenate(recs) if recs else np.zeros(0, dc.MATRIX_DTYPE)


def _choice(name, value, table):
    if value not in table:
        raise ValueError(f"{name} {value!r}: one of {sorted(table)}")
    return table[value]


def _alike(name, ts, dtype, device):
    for k, t in enumerate(ts):
        if t.dtype != dtype or t.device != device:
            raise ValueError(f"{name} {k} is {t.dtype} on {t.device}, expected {dtype} on {device}")


def _check_lr_scale(t, device):
    if t is not None:
        _alike("lr_scale", [t], torch.float32, device)
        if t.numel() != 1:
            raise ValueError(f"lr_scale of {t.numel()} elements, one is needed")


def orthogonalize(grads, steps=5, coeffs=COEFFS, eps=1e-7, hold="pair", out=None, stream=None):
    """Every matrix orthogonalised, in the gradients' dtype: a list of new
    tensors, or `out` (which may be the gradients).  `grads`: a list of
    tensors, or one (then one comes back).  hold: a "pair" of fp16 for each
    value of the steps (about 1e-6 of the result), "one" (1.5e-3 on large
    matrices, a third of the products), or "auto": pairs for float32 and for
    smaller sides under 256, else one."""
    held = _choice("hold", hold, HOLDS)
    one = torch.is_tensor(grads)
    gs = [grads] if one else list(grads)
    if not gs:
        return []
    dt, dev = gs[0].dtype, gs[0].device
    dtype, table = dtype_of(gs[0]), _steps(steps, coeffs)
    _alike("gradient", gs, dt, dev)
    with on(dev, stream):
        if out is None:
            outs = [torch.empty(g.shape, dtype=dt, device=dev) for g in gs]
        else:
            outs = [out] if one else list(out)
            if len(outs) != len(gs):
                raise ValueError(f"{len(outs)} outputs for {len(gs)} gradients")
            _alike("out", outs, dt, dev)
        mats = matrices(gs, outs)
        nbytes = dc.dc_orthogonalize_workspace(dtype, dtype, held, mats, len(mats))
        dc.dc_orthogonalize(dtype, held, mats, len(mats), steps, table, eps, workspace(nbytes, dev), nbytes)
    return outs[0] if one else outs


def update(weights, grads, momentum, lr, mu=0.95, nesterov=True, weight_decay=0.0, scale="rms", steps=5,
           coeffs=COEFFS, eps=1e-7, hold="pair", lr_scale=None, stream=None):
    """One step of the weights and momenta, in place:
      m <- mu m + g;  u = mu m + g (nesterov) or m
      w <- (1 - l weight_decay) w - l s orthogonalize(u)
    with l = lr (times lr_scale, a device float32 read when the work runs) and
    s the shape's factor: "none", "aspect" sqrt(max(1, rows / cols)) or "rms"
    0.2 sqrt(max(rows, cols)).  Lists of tensors, or one of each; momenta are
    float32, weights and gradients each bfloat16 or float32.  hold: as for
    orthogonalize(); "auto" takes pairs for float32 weights too."""
    held, mode = _choice("hold", hold, HOLDS), _choice("scale", scale, SCALES)
    if torch.is_tensor(weights):
        weights, grads, momentum = [weights], [grads], [momentum]
    ws, gs, ms = list(weights), list(grads), list(momentum)
    if not len(ws) == len(gs) == len(ms):
        raise ValueError(f"{len(ws)} weights, {len(gs)} gradients, {len(ms)} momenta")
    if not ws:
        return
    dev = gs[0].device
    dtype, wtype, table = dtype_of(gs[0]), dtype_of(ws[0]), _steps(steps, coeffs)
    _alike("gradient", gs, gs[0].dtype, dev)
    _alike("weight", ws, ws[0].dtype, dev)
    _alike("momentum", ms, torch.float32, dev)
    _check_lr_scale(lr_scale, dev)
    mats = matrices(gs, ws, ms)
    with on(dev, stream):
        nbytes = dc.dc_orthogonalize_workspace(dtype, wtype, held, mats, len(mats))
        dc.dc_muon_update(dtype, wtype, held, mats, len(mats), lr, lr_scale, mu, 1 if nesterov else 0,
                          weight_decay, mode, steps, table, eps, workspace(nbytes, dev), nbytes)

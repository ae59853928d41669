"""The global norm of reduced gradients and clipping by it, on torch tensors.

Between the reduction and the owner's update: grad_norm() and
clip_grad_norm() take a list of tensors of any shapes, bfloat16 and float32
together (Zero1FlushExecutor.clip_gradients and DeferredReducer.clip run them
on what a flush or a deferred reduce wrote).  A job of several processes adds
its squares up: sum_squares() on each, one all-reduce of the double, and
clip_grad_norm(squares=...).

Marshalling only: everything runs in libdc.so (dc_grad_norm, dc_grad_clip) on
`stream`, or on torch's current stream of the tensors' device.  Nothing here
is seen by autograd.
"""
import numpy as np
import torch

from . import dc
from .linear import dtype_of, on, workspace


def _runs(name, t):
    """(rows, cols, row stride) of a tensor's elements in memory, in any order
    of its dimensions."""
    dims = sorted((s, n) for n, s in zip(t.shape, t.stride()) if n > 1)
    if t.numel() == 0:
        return 0, 0, 0
    cols = 1
    while dims and dims[0][0] == cols:
        cols *= dims.pop(0)[1]
    if not dims:
        return 1, cols, cols
    ld, rows = dims.pop(0)
    while dims and dims[0][0] == ld * rows:
        rows *= dims.pop(0)[1]
    if dims or ld < cols:
        raise ValueError(f"{name} of shape {tuple(t.shape)} and strides {t.stride()} is not rows of one stride")
    return rows, cols, ld


def gradients(grads, outs=None):
    """GRADIENT_DTYPE records of lists of tensors, every row counted."""
    recs = np.zeros(len(grads), dc.GRADIENT_DTYPE)
    lists = (grads,) if outs is None else (grads, outs)
    if all(all(map(torch.Tensor.is_contiguous, ts)) for ts in lists):
        # one run each: a list call a field, a tenth of what a tensor at a time costs
        shapes, kinds = [list(map(torch.Tensor.size, ts)) for ts in lists], [[t.dtype for t in ts] for ts in lists]
        codes = {k: dtype_of(t) for k, t in {t.dtype: t for t in grads}.items()}
        if shapes[0] == shapes[-1] and kinds[0] == kinds[-1]:
            recs["grad"] = list(map(torch.Tensor.data_ptr, grads))
            if outs is not None:
                recs["out"] = list(map(torch.Tensor.data_ptr, outs))
            n = np.array(list(map(torch.Tensor.numel, grads)), np.int64)
            recs["cols"] = recs["ld_grad"] = recs["ld_out"] = n
            recs["rows"] = recs["counted"] = n > 0
            recs["dtype"] = [codes[k] for k in kinds[0]]
            return recs
    for k, g in enumerate(grads):
        rows, cols, ld = _runs(f"gradient {k}", g)
        o, ld_out = 0, ld
        if outs is not None:
            t = outs[k]
            if t.shape != g.shape or t.dtype != g.dtype:
                raise ValueError(f"out {k} is {t.dtype} of shape {tuple(t.shape)}, "
                                 f"its gradient {g.dtype} of {tuple(g.shape)}")
            out = _runs(f"out {k}", t)
            if rows == 1 and out[0] > 1:             # the runs of the other one
                rows, cols = out[0], out[1]
                ld = cols
            elif out[0] == 1:
                out = rows, cols, cols
            order = [d for d in range(g.dim()) if g.shape[d] > 1]
            if out[:2] != (rows, cols) or (sorted(order, key=g.stride) != sorted(order, key=t.stride)):
                raise ValueError(f"out {k} of strides {t.stride()} is not laid out as its gradient of {g.stride()}")
            o, ld_out = t.data_ptr(), out[2]
        recs[k] = (g.data_ptr(), o, ld, ld_out, rows, cols, rows, dtype_of(g), 0)
    return recs


def _list(tensors):
    ts = [tensors] if torch.is_tensor(tensors) else list(tensors)
    if not ts:
        raise ValueError("no gradients")
    return ts, _one_device("gradient", ts, ts[0].device)


def _one_device(name, ts, device):
    if set(map(torch.Tensor.get_device, ts)) != {device.index if device.type == "cuda" else -1}:
        for k, t in enumerate(ts):
            if t.device != device:
                raise ValueError(f"{name} {k} on {t.device}, expected {device}")
    return device


def _scalar(name, t, dtype, device):
    if t.dtype != dtype or t.device != device or t.numel() != 1:
        raise ValueError(f"{name} is {t.numel()} of {t.dtype} on {t.device}, expected one {dtype} on {device}")
    return t


def sum_squares(grads, out=None, accumulate=False, stream=None):
    """The sum of every element's square, a float64 scalar tensor: `out`,
    added to with accumulate, or a new one."""
    gs, dev = _list(grads)
    recs = gradients(gs)
    if accumulate and out is None:
        raise ValueError("accumulate needs out")
    with on(dev, stream):
        if out is None:
            out = torch.empty((), dtype=torch.float64, device=dev)
        _scalar("out", out, torch.float64, dev)
        nbytes = dc.dc_grad_clip_workspace()
        dc.dc_grad_norm(recs, len(recs), 1 if accumulate else 0, out, None, workspace(nbytes, dev), nbytes)
    return out


def grad_norm(grads, stream=None):
    """The global norm, a float32 scalar tensor."""
    gs, dev = _list(grads)
    recs = gradients(gs)
    with on(dev, stream):
        norm = torch.empty((), dtype=torch.float32, device=dev)
        nbytes = dc.dc_grad_clip_workspace()
        dc.dc_grad_norm(recs, len(recs), 0, None, norm, workspace(nbytes, dev), nbytes)
    return norm


def clip_grad_norm(grads, max_norm, eps=1e-6, out=None, squares=None, stream=None):
    """Scales every gradient by min(1, max_norm / (norm + eps)), in place or into
    `out` (a list of tensors like them), and returns the norm before, a
    float32 scalar tensor.  A gradient may be in the list once.  squares: a
    float64 scalar to take the norm from instead of the list (sum_squares).
    An infinity gives the factor 0, a NaN makes every gradient NaN: the
    returned norm tells."""
    gs, dev = _list(grads)
    if out is None:
        outs = gs
    else:
        outs = [out] if torch.is_tensor(out) else list(out)
        if len(outs) != len(gs):
            raise ValueError(f"{len(outs)} outputs for {len(gs)} gradients")
        _one_device("out", outs, dev)
    recs = gradients(gs, outs)
    if squares is not None:
        _scalar("squares", squares, torch.float64, dev)
    return clip_records(recs, max_norm, eps, squares, dev, stream)


def clip_records(recs, max_norm, eps, squares, dev, stream):
    with on(dev, stream):
        norm = torch.empty((), dtype=torch.float32, device=dev)
        nbytes = dc.dc_grad_clip_workspace()
        dc.dc_grad_clip(recs, len(recs), squares, max_norm, eps, norm, None, workspace(nbytes, dev), nbytes)
    return norm

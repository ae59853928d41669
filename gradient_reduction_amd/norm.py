"""The norms around a block on torch tensors: the norm after it with its gate
and the residual's scale, and the norm before the next one, in one pass; and
their backward, whose gains' and gates' gradients can be added straight into an
fp32 accumulator.

Marshalling only: everything runs in libdc.so (dc_norm, dc_norm_backward) on
`stream`, or on torch's current stream of the tensors' device; workspaces come
from torch's allocator.  Tensors [..., D] are tokens in order; rows may have
any one stride of at least D.  Nothing here is seen by autograd: backward() is
called by hand.
"""
import math

import torch

from . import dc
from .linear import MOST, _apart, _rows, _span, _vector, dtype_of, on, workspace


def _tokens(name, t, like, T, D, dtype, device):
    """(t [..., D] as T rows, their stride), of `like`'s shape."""
    if t.shape != like:
        raise ValueError(f"{name} of shape {tuple(t.shape)}, expected {tuple(like)}")
    if t.dim() != 2:
        try:
            t = t.view(T, D)
        except RuntimeError:
            raise ValueError(f"{name} of strides {t.stride()} is not rows of one stride") from None
    return _rows(name, t, T, D, dtype, device)


def _gate(name, gate, T, D, dtypes, device):
    """(gate [D] or [rows, D] as rows, their number, their stride)."""
    rows = 1 if gate.dim() == 1 else gate.shape[0] if gate.dim() == 2 else 0
    if rows < 1 or gate.shape[-1] != D or T % rows:
        raise ValueError(f"{name} of shape {tuple(gate.shape)}: [{D}], or rows of it that divide {T} tokens")
    if gate.dtype not in dtypes:
        raise ValueError(f"{name} is {gate.dtype}, expected {dtypes}")
    gate, ld = _rows(name, gate.view(rows, D) if gate.dim() == 1 else gate, rows, D, gate.dtype, device)
    return gate, rows, ld


def _float32(name, v):
    if not abs(v) <= MOST:
        raise ValueError(f"{name} {v} is not finite in float32")


class _Operands:
    """What forward and backward share, checked."""

    def __init__(self, first, gain, h, post_gain, gate, scale, offset, eps):
        if first.dim() < 1:
            raise ValueError("a scalar has no rows")
        self.dt, self.dev, self.like = first.dtype, first.device, first.shape
        self.dtype = dtype_of(first)
        self.T, self.D = first.shape[:-1].numel(), first.shape[-1]
        for name, v in (("scale", scale), ("offset", offset), ("eps", eps)):
            _float32(name, v)
        if eps < 0 or math.isnan(eps):
            raise ValueError(f"eps {eps} < 0")
        if h is None and (post_gain is not None or gate is not None):
            raise ValueError("post_gain and gate need h")
        if h is None and gain is None:
            raise ValueError("gain or h is needed")
        self.h, self.ld_h = (None, 0) if h is None else self.rows("h", h)
        self.gain = None if gain is None else _vector("gain", gain, self.D, (self.dt,), self.dev)
        self.post = None if post_gain is None else _vector("post_gain", post_gain, self.D, (self.dt,), self.dev)
        self.gate, self.gate_rows, self.ld_gate = None, 1, 0
        if gate is not None:
            self.gate, self.gate_rows, self.ld_gate = _gate("gate", gate, self.T, self.D, (self.dt,), self.dev)

    def rows(self, name, t):
        return _tokens(name, t, self.like, self.T, self.D, self.dt, self.dev)

    def empty(self):
        return torch.empty(self.like, dtype=self.dt, device=self.dev)


def forward(x, gain=None, h=None, post_gain=None, gate=None, scale=1.0, offset=0.0, eps=1e-6, out=None, out_norm=None,
            stream=None):
    """(s, y): the residual stream s = x + scale * gate * u after a block with
    output h, u = (offset + post_gain) * h / rms(h), and y = (offset + gain) * s /
    rms(s), the next block's input; rms(v) = sqrt(mean(v^2) + eps) over the last
    dimension.  Without post_gain u is h, without gate it is 1, without h s is x
    itself, without gain y is None.  gate: [D], or [rows, D] with each row for
    an equal share of the tokens in turn.  `out` is for s (x and h are allowed),
    `out_norm` for y."""
    o = _Operands(x, gain, h, post_gain, gate, scale, offset, eps)
    xr, ld_x = o.rows("x", x)
    if (h is None and out is not None) or (gain is None and out_norm is not None):
        raise ValueError("out without h" if out is not None and h is None else "out_norm without gain")
    with on(o.dev, stream):
        s, y = x, None
        sr, ld_s, yr, ld_y = None, 0, None, 0
        if h is not None:
            s = o.empty() if out is None else out
            sr, ld_s = o.rows("out", s)
        if gain is not None:
            y = o.empty() if out_norm is None else out_norm
            yr, ld_y = o.rows("out_norm", y)
        dc.dc_norm(o.dtype, o.T, o.D, xr, ld_x, o.h, o.ld_h, o.post, o.gate, o.gate_rows, o.ld_gate, o.gain, scale,
                   offset, eps, sr, ld_s, yr, ld_y)
    return s, y


def backward(dy, s, gain=None, ds=None, h=None, post_gain=None, gate=None, scale=1.0, offset=0.0, eps=1e-6, dgain=None,
             dpost_gain=None, dgate=None, accumulate=False, need_dx=True, need_dh=True, need_params=True,
             grad_dtype=torch.float32, stream=None):
    """(dx, dh, dgain, dpost_gain, dgate) of forward(), from dy, y's gradient,
    ds, the one that reaches s from later (None: 0), and the s that forward()
    gave (without gain dy may be None).  The parameters' gradients are float32 or x's dtype; given ones are
    written, or added to with accumulate; others are made in grad_dtype, unless
    need_params is unset.  What has no operand is None.  A call that is refused
    has changed nothing."""
    with on(s.device, stream):
        outs, launch = _backward(dy, s, gain, ds, h, post_gain, gate, scale, offset, eps, dgain, dpost_gain, dgate,
                                 accumulate, need_dx, need_dh, need_params, grad_dtype)
        launch()
    return outs


def _backward(dy, s, gain, ds, h, post_gain, gate, scale, offset, eps, dgain, dpost_gain, dgate, accumulate, need_dx,
              need_dh, need_params, grad_dtype):
    """backward()'s checks and allocations, in the caller's on(): (its outputs,
    what launches it).  Nothing is refused after the first launch."""
    o = _Operands(s, gain, h, post_gain, gate, scale, offset, eps)
    sr, ld_s = o.rows("s", s)
    dyr, ld_dy, dsr, ld_ds = None, 0, None, 0
    if gain is not None:
        if dy is None:
            raise ValueError("gain needs dy")
        dyr, ld_dy = o.rows("dy", dy)
    if ds is not None:
        dsr, ld_ds = o.rows("ds", ds)
    grads, spans, kinds, ld_dgate = [], [], set(), 0
    size = s.element_size()
    reads = [_span("h", o.h, o.T, o.D, o.ld_h, size)] if h is not None else []
    if gain is not None:
        reads += [_span("dy", dyr, o.T, o.D, ld_dy, size), _span("s", sr, o.T, o.D, ld_s, size),
                  _span("gain", o.gain, 1, o.D, o.D, size)]
    if ds is not None:
        reads.append(_span("ds", dsr, o.T, o.D, ld_ds, size))
    if post_gain is not None:
        reads.append(_span("post_gain", o.post, 1, o.D, o.D, size))
    if gate is not None:
        reads.append(_span("gate", o.gate, o.gate_rows, o.D, o.ld_gate, size))
    for name, operand, given in (("dgain", gain, dgain), ("dpost_gain", post_gain, dpost_gain), ("dgate", gate, dgate)):
        if given is not None and operand is None:
            raise ValueError(f"{name} without its operand")
        if operand is None or (given is None and not need_params):
            grads.append(None)
            continue
        if given is None:
            if accumulate:
                raise ValueError(f"accumulate needs {name}")
            given = torch.empty(operand.shape, dtype=grad_dtype, device=o.dev)
        if name == "dgate":
            if given.shape != gate.shape:
                raise ValueError(f"dgate of shape {tuple(given.shape)}, expected {tuple(gate.shape)}")
            rows, n, ld_dgate = _gate(name, given, o.T, o.D, (torch.float32, o.dt), o.dev)
            at = _span(name, rows, n, o.D, ld_dgate, given.element_size())
        else:
            _vector(name, given, o.D, (torch.float32, o.dt), o.dev)
            at = _span(name, given, 1, o.D, o.D, given.element_size())
        _apart(at, reads + spans)
        spans.append(at)
        kinds.add(given.dtype)
        grads.append(given)
    if len(kinds) > 1:
        raise ValueError(f"the parameters' gradients are {sorted(map(str, kinds))}: one dtype is needed")
    grad = dtype_of(next(g for g in grads if g is not None)) if kinds else dc.DC_F32
    nbytes = dc.dc_norm_backward_workspace(o.dtype, o.T, o.D, o.gate_rows)
    dx = o.empty() if need_dx else None
    dh = o.empty() if need_dh and h is not None else None
    wanted = (need_dx or dh is not None or kinds) and (o.T or kinds)
    ws = workspace(nbytes, o.dev) if wanted else None

    def launch():
        if wanted:
            dc.dc_norm_backward(o.dtype, o.T, o.D, dyr, ld_dy, dsr, ld_ds, sr if gain is not None else None, ld_s, o.h,
                                o.ld_h, o.post, o.gate, o.gate_rows, o.ld_gate, o.gain, scale, offset, eps, dx, o.D,
                                dh, o.D, grad, grads[0], grads[1], grads[2], ld_dgate, 1 if accumulate else 0, ws,
                                nbytes)

    return (dx, dh, *grads), launch

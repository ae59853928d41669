"""A linear layer's products on torch tensors: forward with bias, activation
and residual in the product's epilogue, and its backward, whose weight
gradient can be added straight into an fp32 accumulator.

Marshalling only: shapes, dtypes and devices are checked, outputs and
workspaces come from torch's allocator, and everything runs in libdc.so
(dc_linear, dc_bias_act_backward, dc_linear_backward) on `stream`, or on
torch's current stream of the tensors' device.  Rows may have any stride of at
least their length; columns are contiguous.  Tensors made on another stream
are the caller's to order, as in torch.  Nothing here is seen by autograd:
backward() is called by hand.
"""
import contextlib

import torch

from . import dc

ACTS = {"none": dc.DC_ACT_NONE, "relu": dc.DC_ACT_RELU, "gelu": dc.DC_ACT_GELU, "silu": dc.DC_ACT_SILU}
_DTYPES = {torch.bfloat16: dc.DC_BF16, torch.float32: dc.DC_F32}


def dtype_of(t) -> int:
    if t.dtype not in _DTYPES:
        raise ValueError(f"dtype {t.dtype}: bfloat16 or float32 is needed")
    return _DTYPES[t.dtype]


def on(device, stream):
    """The context in which a call on `device` allocates and launches."""
    if device.type != "cuda":
        raise ValueError(f"tensors on {device}: a GPU is needed")
    if stream is not None:
        if isinstance(stream, int):
            stream = torch.cuda.ExternalStream(stream, device=device)
        if stream.device != device:
            raise ValueError(f"stream of {stream.device}, tensors on {device}")
        return torch.cuda.stream(stream)
    if device.index == torch.cuda.current_device():
        return contextlib.nullcontext()
    return torch.cuda.device(device)


def workspace(nbytes: int, device):
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def _rows(name, t, rows, cols, dtype, device):
    """(tensor, row stride) of a [rows, cols] operand."""
    if t.dim() != 2 or t.shape[0] != rows or t.shape[1] != cols:
        raise ValueError(f"{name} of shape {tuple(t.shape)}, expected {(rows, cols)}")
    if t.dtype != dtype:
        raise ValueError(f"{name} is {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name} on {t.device}, expected {device}")
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"{name}: columns must be contiguous (strides {t.stride()})")
    if rows > 1 and t.stride(0) < cols:
        raise ValueError(f"{name}: rows overlap (strides {t.stride()})")
    return t, t.stride(0) if rows > 1 else cols


def _vector(name, t, n, dtypes, device):
    if t.dim() != 1 or t.shape[0] != n or (n > 1 and t.stride(0) != 1):
        raise ValueError(f"{name} of shape {tuple(t.shape)} and strides {t.stride()}, expected {n} contiguous")
    if t.dtype not in dtypes or t.device != device:
        raise ValueError(f"{name} is {t.dtype} on {t.device}, expected {dtypes} on {device}")
    return t


def _act(act):
    if act not in ACTS:
        raise ValueError(f"act {act!r}: one of {sorted(ACTS)}")
    return ACTS[act]


def _sizes(x, w):
    if x.dim() != 2 or w.dim() != 2:
        raise ValueError(f"x {tuple(x.shape)} and w {tuple(w.shape)} must be matrices")
    return x.shape[0], w.shape[0], w.shape[1]


def forward(x, w, bias=None, residual=None, act="none", save_pre=False, out=None, pre=None, stream=None):
    """act(x wT + bias) + residual for x [T, K] and w [N, K]; with save_pre
    (or `pre`, a tensor for it) also the pre-activation x wT + bias, which
    bias_act_backward reads: (y, pre).  `out` may be `residual`."""
    T, N, K = _sizes(x, w)
    code, dt, dev = _act(act), x.dtype, x.device
    dtype = dtype_of(x)
    x, ld_x = _rows("x", x, T, K, dt, dev)
    w, ld_w = _rows("w", w, N, K, dt, dev)
    if bias is not None:
        _vector("bias", bias, N, (dt,), dev)
    ld_res = 0
    if residual is not None:
        residual, ld_res = _rows("residual", residual, T, N, dt, dev)
    with on(dev, stream):
        if out is None:
            out = torch.empty((T, N), dtype=dt, device=dev)
        if pre is None and save_pre:
            pre = torch.empty((T, N), dtype=dt, device=dev)
        out, ld_y = _rows("out", out, T, N, dt, dev)
        ld_pre = 0
        if pre is not None:
            pre, ld_pre = _rows("pre", pre, T, N, dt, dev)
        nbytes = dc.dc_linear_workspace(dtype, T, N, K)
        dc.dc_linear(dtype, T, N, K, x, ld_x, w, ld_w, bias, residual, ld_res, code, pre, ld_pre, out,
                     ld_y, workspace(nbytes, dev), nbytes)
    return out if pre is None else (out, pre)


def _span(name, t, rows, cols, ld, size):
    """Where an operand of `size`-byte elements lies: (name, first byte, end,
    bytes of a row, bytes from row to row, rows)."""
    p, step = t.data_ptr(), ld * size
    return name, p, p + (rows - 1) * step + cols * size, cols * size, step, rows


def _apart(out, ins):
    """Refuses a written operand (a _span) that shares an element with one of
    the others.  Between rows of one stride there may be others' columns, or a
    vector."""
    name, pa, end_a, ca, step_a, ra = out
    for other, pb, end_b, cb, step_b, rb in ins:
        if pa >= end_b or pb >= end_a or not ra or not rb:
            continue
        step = step_a if rb == 1 else step_b
        d = (pb - pa) % step
        if (ra > 1 and rb > 1 and step_a != step_b) or d < ca or d + cb > step:
            raise ValueError(f"{name} and {other} overlap")


def _bias_act(dy, pre, act, dz, db, accumulate, need_dz, need_db, grad_dtype):
    """bias_act_backward's checks and allocations, in the caller's on():
    (dz, db, what launches it)."""
    if dy.dim() != 2:
        raise ValueError(f"dy {tuple(dy.shape)} must be a matrix")
    T, N = dy.shape
    code, dt, dev = _act(act), dy.dtype, dy.device
    dtype = dtype_of(dy)
    dy, ld_dy = _rows("dy", dy, T, N, dt, dev)
    ld_pre = 0
    if code != dc.DC_ACT_NONE:
        if pre is None:
            raise ValueError(f"act {act!r} needs the pre-activation")
        pre, ld_pre = _rows("pre", pre, T, N, dt, dev)
    else:
        pre = None
        if need_dz and dz is None:
            dz, need_dz = dy, False
    if accumulate and db is None:
        raise ValueError("accumulate needs db")
    if need_dz and dz is None:
        dz = torch.empty((T, N), dtype=dt, device=dev)
    if db is None and need_db:
        db = torch.empty(N, dtype=grad_dtype, device=dev)
    if db is not None:
        _vector("db", db, N, (torch.float32, dt), dev)
    ld_dz = 0
    if need_dz:
        dz, ld_dz = _rows("dz", dz, T, N, dt, dev)
    if not ((need_dz and T) or db is not None):
        return dz, db, lambda: None
    nbytes = dc.dc_bias_act_workspace(dtype, T, N) if db is not None else 0
    ws = workspace(nbytes, dev)

    def launch():
        dc.dc_bias_act_backward(dtype, T, N, dy, ld_dy, pre, ld_pre, code, dz if need_dz else None,
                                ld_dz, dtype_of(db) if db is not None else dc.DC_F32, db,
                                1 if accumulate else 0, ws, nbytes)

    return dz, db, launch


def bias_act_backward(dy, pre=None, act="none", dz=None, db=None, accumulate=False, need_dz=True,
                      need_db=False, grad_dtype=torch.float32, stream=None):
    """(dz, db): dz = dy act'(pre) and the bias gradient, its column sums
    (added to `db` with accumulate).  db is returned when it is given or
    need_db is set; dz when need_dz is set, and is dy itself without an
    activation."""
    with on(dy.device, stream):
        dz, db, launch = _bias_act(dy, pre, act, dz, db, accumulate, need_dz, need_db, grad_dtype)
        launch()
    return dz, db


def backward(dy, x, w, pre=None, act="none", dw=None, db=None, accumulate=False, need_dx=True,
             need_dw=True, grad_dtype=torch.float32, stream=None):
    """(dx, dw, db) of forward() from dy, the gradient of y; the residual's
    gradient is dy.  dw [N, K] and db [N] are float32 or x's dtype; given ones
    are written, or added to with accumulate; db only when given.  They may
    share no element with each other, x or w, nor db with dy or pre.  dz = dy act'(pre)
    is rounded once to x's dtype on its way into the products.  A call that is
    refused has changed nothing."""
    with on(x.device, stream):
        dx, dw, db, launch = _backward(dy, x, w, pre, act, dw, db, accumulate, need_dx, need_dw, grad_dtype)
        launch()
    return dx, dw, db


def _backward(dy, x, w, pre, act, dw, db, accumulate, need_dx, need_dw, grad_dtype=torch.float32):
    """backward()'s checks and allocations, in the caller's on(): (dx, dw, db,
    what launches it).  Nothing is refused after the first launch."""
    T, N, K = _sizes(x, w)
    dt, dev = x.dtype, x.device
    dtype = dtype_of(x)
    x, ld_x = _rows("x", x, T, K, dt, dev)
    w, ld_w = _rows("w", w, N, K, dt, dev)
    dy, ld_dy = _rows("dy", dy, T, N, dt, dev)
    if accumulate and need_dw and dw is None:
        raise ValueError("accumulate needs dw")
    ld_dw, dw_type, given = 0, dc.DC_F32, dw is not None and need_dw
    if need_dw:
        if dw is None:
            dw = torch.empty((N, K), dtype=grad_dtype, device=dev)
        if dw.dtype not in (torch.float32, dt):
            raise ValueError(f"dw is {dw.dtype}, expected float32 or {dt}")
        dw, ld_dw = _rows("dw", dw, N, K, dw.dtype, dev)
        dw_type = dtype_of(dw)
    else:
        dw = None
    elementwise = lambda: None                                           # noqa: E731
    dz = dy
    if act != "none" or db is not None:
        dz, db, elementwise = _bias_act(dy, pre, act, None, db, accumulate and db is not None, True, False,
                                        grad_dtype)
    if given or db is not None:
        size = 2 if dtype == dc.DC_BF16 else 4
        grads = [_span("dw", dw, N, K, ld_dw, 2 if dw_type == dc.DC_BF16 else 4)] if given else []
        products = [_span("x", x, T, K, ld_x, size)] if need_dw else []
        if need_dx:
            products.append(_span("w", w, N, K, ld_w, size))
        first = [_span("dy", dy, T, N, ld_dy, size)]
        if given:       # dy and pre are read before it is written, unless dy is dz
            _apart(grads[0], products + first if act == "none" else products)
        if db is not None:
            if act != "none":
                first.append(_span("pre", pre, T, N, pre.stride(0) if T > 1 else N, size))
            _apart(_span("db", db, 1, N, N, db.element_size()), products + first + grads)
    dz, ld_dz = _rows("dz", dz, T, N, dt, dev)
    dx = torch.empty((T, K), dtype=dt, device=dev) if need_dx else None
    any_product = (need_dx and T) or need_dw
    nbytes = dc.dc_linear_backward_workspace(dtype, T, N, K) if any_product else 0
    ws = workspace(nbytes, dev)

    def launch():
        elementwise()
        if any_product:
            dc.dc_linear_backward(dtype, T, N, K, dz, ld_dz, w, ld_w, x, ld_x, dx, K, dw_type, dw, ld_dw,
                                  1 if accumulate else 0, ws, nbytes)

    return dx, dw, db, launch

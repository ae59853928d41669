"""An embedding on torch tensors: the lookup with scaling, and its table's
gradient by sorted tokens, which can be added straight into an fp32
accumulator.

Marshalling only: everything runs in libdc.so (dc_embedding,
dc_embedding_backward) on `stream`, or on torch's current stream of the
tensors' device; workspaces come from torch's allocator.  Ids are int32 or
int64; one outside the table (padding, a token of another rank's part) gives
a row of zeros and no gradient.  Nothing here is seen by autograd: backward()
is called by hand.
"""
import torch

from . import dc
from .linear import MOST, _apart, _rows, _span, dtype_of, on, workspace

_IDS = {torch.int32: 4, torch.int64: 8}


def _id_bytes(ids, device) -> int:
    if ids.dtype not in _IDS:
        raise ValueError(f"ids are {ids.dtype}: int32 or int64 is needed")
    if ids.device != device:
        raise ValueError(f"ids on {ids.device}, expected {device}")
    return _IDS[ids.dtype]


def _check_scale(scale):
    if not abs(scale) <= MOST:
        raise ValueError(f"scale {scale} is not finite in float32")


def _tokens(name, t, ids, D):
    """t [*ids.shape, D] as rows of one stride."""
    if tuple(t.shape) != tuple(ids.shape) + (D,):
        raise ValueError(f"{name} of shape {tuple(t.shape)}, expected {tuple(ids.shape) + (D,)}")
    if t.dim() == 2:
        return t
    try:
        return t.view(ids.numel(), D)
    except RuntimeError:
        raise ValueError(f"{name} of strides {t.stride()} is not rows of one stride") from None


def forward(ids, table, scale=1.0, out=None, stream=None):
    """scale * table[ids] for ids of any shape and a table [rows, D]: a tensor
    [*ids.shape, D] in the table's dtype, or `out`."""
    if table.dim() != 2:
        raise ValueError(f"table {tuple(table.shape)} must be a matrix")
    rows, D = table.shape
    _check_scale(scale)
    dt, dev = table.dtype, table.device
    dtype, size, T = dtype_of(table), _id_bytes(ids, dev), ids.numel()
    table, ld_table = _rows("table", table, rows, D, dt, dev)
    with on(dev, stream):
        if out is None:
            out = torch.empty(tuple(ids.shape) + (D,), dtype=dt, device=dev)
        flat, ld_out = _rows("out", _tokens("out", out, ids, D), T, D, dt, dev)
        dc.dc_embedding(dtype, size, T, rows, D, ids.contiguous(), table, ld_table, scale, flat, ld_out)
    return out


def backward(dy, ids, rows=None, scale=1.0, dtable=None, accumulate=False, grad_dtype=torch.float32, stream=None):
    """The gradient of the table [rows, D] from dy [*ids.shape, D], that of
    forward(): `dtable`, written, or added to with accumulate, in float32 or
    dy's dtype, or a new tensor in grad_dtype."""
    with on(dy.device, stream):
        dtable, launch = _backward(dy, ids, rows, scale, dtable, accumulate, grad_dtype)
        launch()
    return dtable


def _backward(dy, ids, rows, scale, dtable, accumulate, grad_dtype):
    """backward()'s checks and allocations, in the caller's on(): (dtable, what
    launches it).  Nothing is refused after the first launch."""
    if dy.dim() < 1:
        raise ValueError("dy is a scalar")
    dt, dev, D, T = dy.dtype, dy.device, dy.shape[-1], ids.numel()
    dtype, size = dtype_of(dy), _id_bytes(ids, dev)
    dy, ld_dy = _rows("dy", _tokens("dy", dy, ids, D), T, D, dt, dev)
    _check_scale(scale)
    if rows is None and dtable is None:
        raise ValueError("rows or dtable is needed")
    if dtable is not None and dtable.dim() != 2:
        raise ValueError(f"dtable {tuple(dtable.shape)} must be a matrix")
    rows = dtable.shape[0] if rows is None else rows
    if dtable is None:
        if accumulate:
            raise ValueError("accumulate needs dtable")
        dtable = torch.empty((rows, D), dtype=grad_dtype, device=dev)
    if dtable.dtype not in (torch.float32, dt):
        raise ValueError(f"dtable is {dtable.dtype}, expected float32 or {dt}")
    dtable, ld = _rows("dtable", dtable, rows, D, dtable.dtype, dev)
    ids = ids.contiguous()
    _apart(_span("dtable", dtable, rows, D, ld, dtable.element_size()),
           [_span("dy", dy, T, D, ld_dy, dy.element_size()), _span("ids", ids, 1 if T else 0, T, T, size)])
    nbytes = dc.dc_embedding_backward_workspace(dtype, T, rows, D)
    ws = workspace(nbytes, dev)

    def launch():
        dc.dc_embedding_backward(dtype, size, T, rows, D, dy, ld_dy, ids, scale, dtype_of(dtable), dtable, ld,
                                 1 if accumulate else 0, ws, nbytes)

    return dtable, launch

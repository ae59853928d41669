"""Gradient accumulation with the data-parallel reduce deferred to update().

MaxText PR "Defer the data-parallel gradient all-reduce to update() under
gradient accumulation": each replica accumulates its own micro-batch
gradients locally (What), and one cross-replica reduce runs at update() on the
accumulated sums instead of one per micro-batch; the accumulator lives across
the micro-batches of a step and can be saved and restored mid-step
(What else had to change, accumulator lifetime).

W replicas are the rows of [W, ld] fp32 slabs on one GPU.  Marshalling only:
every step runs in libdc.so (dc_accumulate, dc_deferred_reduce,
dc_accumulate_reduce); torch supplies the memory and the stream.

A micro-batch comes either whole, as a slab of gradients (accumulate), or
layer by layer as the products that make them (accumulate_linear and its
like, then end_micro_batch): a weight's gradient is then added to its
replica's row by the product itself (dc_linear_backward,
dc_embedding_backward, dc_norm_backward) and never stored on its own.  clip() takes the reduced
gradients' global norm (dc_grad_clip).
"""
from . import dc


class DeferredReducer:
    def __init__(self, W: int, M: int, ld: int = 0, device: str = "cuda"):
        """W replicas of M fp32 gradient elements each; the accumulator is a
        [W, ld] slab (ld defaults to M rounded up to 64 elements)."""
        import torch
        self.torch = torch
        self.W, self.M = W, M
        self.ld = ld if ld else max(64, -(-M // 64) * 64)
        if self.ld < M:
            raise ValueError(f"ld={self.ld} < M={M}")
        self.acc = torch.empty((W, self.ld), dtype=torch.float32, device=device)
        self.micro_batches = 0
        self.open = False          # a micro-batch is being added layer by layer
        self.stale = set()         # rows that still hold what was there before this step

    def accumulate(self, x, ld_x: int, stream=None) -> None:
        """Add one micro-batch: acc[r] += x[r] on every replica row (the first
        micro-batch of a step starts from +0)."""
        self._closed("accumulate()")
        self._clear_stale(stream)
        dc.dc_accumulate(self.W, x, ld_x, self.acc, self.ld, self.M, 1 if self.micro_batches == 0 else 0,
                         stream)
        self.micro_batches += 1

    def _closed(self, what):
        if self.open:
            raise RuntimeError(f"{what} inside a micro-batch: call end_micro_batch() first")

    def _clear_stale(self, stream=None):
        """Rows of a step's replicas that had no layer yet."""
        if self.stale:
            from . import linear
            with linear.on(self.acc.device, stream):
                for r in sorted(self.stale):
                    self.acc[r].zero_()
            self.stale = set()

    def _place(self, row, offset, n):
        if not 0 <= row < self.W:
            raise ValueError(f"row {row} outside [0, {self.W})")
        if offset < 0 or offset + n > self.M:
            raise ValueError(f"elements [{offset}, {offset + n}) outside [0, {self.M})")
        return self.acc[row, offset:offset + n]

    def accumulate_linear(self, row: int, offset: int, dy, x, w, pre=None, act: str = "none",
                          bias_offset=None, need_dx: bool = True, stream=None):
        """The backward of one linear layer of replica `row` (linear.backward):
        its weight gradient [N, K] is added at elements offset .. offset + N K
        of the row and its bias gradient at bias_offset, if given; returns dx
        (None without need_dx).  A parameter used by several layers is given
        once for each.  A replica's first call of a step clears its row, on
        that call's stream, and no call touches another replica's: replicas may
        be on streams of their own.  The caller orders calls of one row, and
        what uses all rows (reduce, accumulate, state_dict) after them."""
        from . import linear
        n, k = w.shape
        dw = self._place(row, offset, n * k).view(n, k)
        db = self._place(row, bias_offset, n) if bias_offset is not None else None
        if bias_offset is not None and bias_offset < offset + n * k and offset < bias_offset + n:
            raise ValueError("the weight's and the bias's elements overlap")
        with linear.on(self.acc.device, stream):
            dx, _, _, launch = linear._backward(dy, x, w, pre, act, dw, db, True, need_dx, True)
            self._add(row, launch)
        return dx

    def _add(self, row, launch):
        """An accepted layer's launches into a row, cleared before its first of a
        step."""
        stale = self.stale if self.open or self.micro_batches else set(range(self.W))
        if row in stale:
            self.acc[row].zero_()
        launch()
        self.stale = stale - {row}
        self.open = True

    def accumulate_embedding(self, row: int, offset: int, dy, ids, rows: int, scale: float = 1.0,
                             stream=None) -> None:
        """The gradient of replica `row`'s embedding table [rows, D], from the
        gradient dy [..., D] of its lookup of `ids` (embedding.backward), added at
        elements offset .. offset + rows D of the row; otherwise as
        accumulate_linear.  A table that is the output's too is given to both."""
        from . import embedding, linear
        if dy.dim() < 1 or rows < 1:
            raise ValueError(f"dy of shape {tuple(dy.shape)} for a table of {rows} rows")
        dtable = self._place(row, offset, rows * dy.shape[-1]).view(rows, dy.shape[-1])
        with linear.on(self.acc.device, stream):
            _, launch = embedding._backward(dy, ids, rows, scale, dtable, True, None)
            self._add(row, launch)

    def accumulate_norm(self, row: int, dy, s, gain=None, ds=None, h=None, post_gain=None, gate=None,
                        scale: float = 1.0, offset: float = 0.0, eps: float = 1e-6, gain_at=None, post_gain_at=None,
                        gate_at=None, need_dx: bool = True, need_dh: bool = True, stream=None):
        """The backward of the norms around a block of replica `row`
        (norm.backward): the gradients of gain [D], post_gain [D] and gate
        ([rows, D] or [D]) are added at elements gain_at, post_gain_at and gate_at
        of the row, where given; returns (dx, dh).  Otherwise as accumulate_linear."""
        from . import linear, norm

        def place(name, operand, at):
            if at is None:
                return None
            if operand is None:
                raise ValueError(f"{name}_at without {name}")
            return self._place(row, at, operand.numel()).view(operand.shape)

        self._place(row, 0, 0)
        grads = [place("gain", gain, gain_at), place("post_gain", post_gain, post_gain_at), place("gate", gate, gate_at)]
        with linear.on(self.acc.device, stream):
            (dx, dh, *_), launch = norm._backward(dy, s, gain, ds, h, post_gain, gate, scale, offset, eps, *grads,
                                                  any(g is not None for g in grads), need_dx, need_dh, False, None)
            self._add(row, launch)
        return dx, dh

    def end_micro_batch(self) -> None:
        """Every layer of every replica's micro-batch has been added."""
        if not self.open:
            raise RuntimeError("end_micro_batch() before any layer")
        self.open = False
        self.micro_batches += 1

    def reduce(self, out, ld_out: int, out_rows: int = 1, last=None, ld_last: int = 0,
               keep_acc: bool = False, stream=None) -> None:
        """update(): the cross-replica fold of the accumulators into
        out[0..out_rows) (1: one reduced copy, W: every replica gets it).
        With `last`, that final micro-batch is accumulated in the same pass
        (dc_accumulate_reduce); keep_acc also writes it to the accumulator.
        The next accumulate() starts a new step."""
        self._closed("reduce()")
        if last is None and self.micro_batches == 0:
            raise RuntimeError("reduce() before any accumulate() in this step")
        self._clear_stale(stream)
        if last is None:
            dc.dc_deferred_reduce(self.W, self.acc, self.ld, out, ld_out, self.M, out_rows, stream)
        else:
            dc.dc_accumulate_reduce(self.W, last, ld_last, self.acc, self.ld,
                                    1 if self.micro_batches == 0 else 0, 1 if keep_acc else 0, out,
                                    ld_out, out_rows, self.M, stream)
        self.micro_batches = 0

    def clip(self, out, ld_out: int, max_norm: float, out_rows: int = 1, eps: float = 1e-6, stream=None):
        """After reduce(), on its stream: scales the reduced gradients in
        out[0..out_rows) by min(1, max_norm / (norm + eps)) and returns their global
        norm before, a float32 scalar tensor; every row holds the same sums, the
        norm counts the first."""
        from . import clip
        import numpy as np
        if out_rows not in (1, self.W):
            raise ValueError(f"out_rows={out_rows}: 1 or W={self.W}")
        if ld_out < self.M:
            raise ValueError(f"ld_out={ld_out} < M={self.M}")
        if not isinstance(out, int):
            have = out.untyped_storage().nbytes() // 4 - out.storage_offset()
            if out.dtype != self.torch.float32 or out.device != self.acc.device or \
                    (out_rows - 1) * ld_out + self.M > have:
                raise ValueError(f"out {tuple(out.shape)} of {out.dtype} on {out.device} with ld_out={ld_out} "
                                 f"does not hold {out_rows} rows of {self.M}")
        at = out if isinstance(out, int) else out.data_ptr()
        rec = np.zeros(1, dc.GRADIENT_DTYPE)
        rec[0] = (at, at, ld_out, ld_out, out_rows, self.M, 1, dc.DC_F32, 0)
        return clip.clip_records(rec, max_norm, eps, None, self.acc.device, stream)

    def state_dict(self) -> dict:
        """The accumulator's state mid-step: a copy of the slab's M columns
        and the micro-batch count."""
        self._closed("state_dict()")
        self._clear_stale()
        return {"acc": self.acc[:, :self.M].clone(), "micro_batches": self.micro_batches}

    def load_state_dict(self, state: dict) -> None:
        acc = state["acc"]
        if tuple(acc.shape) != (self.W, self.M):
            raise ValueError(f"accumulator of shape {tuple(acc.shape)}, expected {(self.W, self.M)}")
        self.acc[:, :self.M].copy_(acc)
        self.open = False
        self.stale = set()
        self.micro_batches = int(state["micro_batches"])

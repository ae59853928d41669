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
layer by layer as the products that make them (accumulate_linear, then
end_micro_batch): a weight's gradient is then added to its replica's row by
the product itself (dc_linear_backward) and never stored on its own.
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
            stale = self.stale if self.open or self.micro_batches else set(range(self.W))
            if row in stale:                                  # the layer is accepted
                self.acc[row].zero_()
            launch()
        self.stale = stale - {row}
        self.open = True
        return dx

    def end_micro_batch(self) -> None:
        """Every layer of every replica's micro-batch has been added."""
        if not self.open:
            raise RuntimeError("end_micro_batch() before any accumulate_linear()")
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

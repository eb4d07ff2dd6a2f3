"""Products grouped by expert, forward and backward (include/waste_train.h: waste_group_forward,
waste_group_backward): each row of a batch against the 16-bit matrix of its expert, the rows sorted by expert.

The routed experts are trained in this form before their matrices are encoded (``waste_rvq_train``), or served in it
where 3 bits are not wanted.  All computation is in the library's kernels.
"""
from __future__ import annotations

import torch

from . import binding as B
from .dense import ACT, check, make, require


class GroupedLinear:
    """w [E, n, k], bf16 or fp16, contiguous on one GPU (borrowed, not copied).  offsets [E + 1] int32 on that GPU:
    the rows of expert e are offsets[e] .. offsets[e + 1] - 1; they are not read by the host.  They may not fall and
    lie within 0 .. rows (``binding.waste_dense_status`` raises afterwards where they did not); rows outside
    offsets[0] .. offsets[E] - 1 are left as they were.  There is no workspace: calls may run at the same time.
    stream: a torch.cuda.Stream, an integer handle or None for the current stream; ordering the tensors' use between
    streams is the caller's."""

    def __init__(self, w: torch.Tensor):
        require(isinstance(w, torch.Tensor) and w.dim() == 3 and w.device.type == "cuda"
                and w.dtype in (torch.bfloat16, torch.float16), "w is a bf16 or fp16 [E, n, k] tensor on a GPU")
        E, n, k = w.shape
        dev, t = w.device, w.dtype
        check(w, "w", (E, n, k), (t,), dev)
        self.w = w
        self.E, self.n, self.k, self.dtype, self.device, self.index = E, n, k, t, dev, dev.index
        self._own, self._out = (t,), (t, torch.float32)
        self.cfg = B.waste_group_config(B.ABI_VERSION, E, k, n, ACT[t])

    def _given(self, x, name, cols, offsets) -> int:
        if not isinstance(x, torch.Tensor) or x.dim() != 2:
            require(False, f"{name}: a [rows, {cols}] tensor is needed")
        check(x, name, (x.shape[0], cols), self._own, self.device)
        check(offsets, "offsets", (self.E + 1,), (torch.int32,), self.device)
        return x.shape[0]

    def forward(self, x, offsets, out=None, mode: int = 0, stream=None):
        """out [rows, n] (fp32 or w's type; made if None) = (mode 0) or += (mode 1) each row of x [rows, k] times
        its expert's matrix, x_r w_e^T."""
        index = self.index
        if B.device_now() != index:
            with torch.cuda.device(index):
                return self.forward(x, offsets, out, mode, stream)
        rows = self._given(x, "x", self.k, offsets)
        if out is None:
            require(mode == 0, "mode 1 adds to a given out")
            out = make((rows, self.n), self.dtype, self.device, stream)
        check(out, "out", (rows, self.n), self._out, self.device)
        B.waste_group_forward(self.cfg, x, rows, offsets, self.w, out, ACT[out.dtype], mode, B.stream_on(index, stream))
        return out

    def backward(self, dy, x, offsets, dx=None, dw=None, accumulate: bool = False, stream=None):
        """Gradients for dy [rows, n]: into dx [rows, k] = dy_r w_e (None: not computed) and dw [E, n, k] = the sum over
        e's rows of dy_r^T x_r (None: not computed; fp32 or w's type; zeros for an expert without rows), added to
        what is there with accumulate.  x may be None where dw is."""
        index = self.index
        if B.device_now() != index:
            with torch.cuda.device(index):
                return self.backward(dy, x, offsets, dx, dw, accumulate, stream)
        rows = self._given(dy, "dy", self.n, offsets)
        if x is not None or dw is not None:
            check(x, "x", (rows, self.k), self._own, self.device)
        if dx is not None:
            check(dx, "dx", (rows, self.k), self._own, self.device)
        gt = self.dtype
        if dw is not None:
            check(dw, "dw", self.w.shape, self._out, self.device)
            gt = dw.dtype
        B.waste_group_backward(self.cfg, dy, x, rows, offsets, self.w, dx, dw, ACT[gt], int(accumulate),
                               B.stream_on(index, stream))

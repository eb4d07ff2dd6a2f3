"""Layer norm over the rows of a matrix, forward and backward (include/waste_train.h: waste_norm_forward,
waste_norm_backward): the norm in front of the router and the experts, with the weight and bias that training gives
it.  All computation is in the library's kernels.
"""
from __future__ import annotations

import torch

from . import binding as B
from .dense import ACT, Workspace, check, make, require

_FLOATS = (torch.float32, torch.bfloat16, torch.float16)
_F32 = (torch.float32,)


class LayerNorm:
    """y = (x - mean) rstd w + b over the last of x's two dimensions.  weight [d], bias [d] or None: fp32, bf16 or
    fp16, of one type, contiguous on one GPU (borrowed, not copied).  The backward's workspace belongs to this object:
    backward calls of one object must not run at the same time on two streams (from several host threads on one
    stream they may), two captured graphs that may replay at the same time need an object each, and an object
    outlives the graphs that hold its calls.  stream: a torch.cuda.Stream, an integer handle (then the object must
    outlive the call) or None for the current stream; ordering the tensors' use between streams is the caller's."""

    def __init__(self, weight: torch.Tensor, bias: torch.Tensor | None = None, eps: float = 1e-5):
        dev, t = weight.device, weight.dtype
        require(dev.type == "cuda" and dev.index is not None and t in _FLOATS and weight.dim() == 1,
                "weight is a [d] tensor of fp32, bf16 or fp16 on a GPU")
        d = weight.shape[0]
        check(weight, "weight", (d,), (t,), dev)
        if bias is not None:
            check(bias, "bias", (d,), (t,), dev)
        self.weight, self.bias, self.eps = weight, bias, float(eps)
        self.d, self.dtype, self.device, self.index = d, t, dev, dev.index
        self._cfg = {}
        self._ws = {}  # the backward's workspace, once it is made
        B.waste_norm_workspace(self._config(t, t), 1)  # refuses a bad d or eps here

    def _config(self, x, y):
        """For x and y of two types."""
        c = self._cfg.get((x, y))
        if c is None:
            c = self._cfg[x, y] = B.waste_norm_config(B.ABI_VERSION, self.d, ACT[x], ACT[y], ACT[self.dtype], self.eps)
        return c

    def __getstate__(self):  # configurations are made anew, a copy's workspace too
        return {**self.__dict__, "_cfg": {}, "_ws": {}}

    def _rows(self, t, name, T=None) -> int:
        """The row stride of a [T, d] tensor whose rows are contiguous."""
        if not (isinstance(t, torch.Tensor) and t.dim() == 2 and t.shape[1] == self.d and (T is None or t.shape[0] == T)
                and t.dtype in ACT and t.device == self.device and (t.shape[0] == 0 or self.d == 1 or t.stride(1) == 1)):
            require(False, f"{name}: a [{'T' if T is None else T}, {self.d}] tensor with contiguous rows, fp32, bf16 or fp16, "
                           f"on {self.device} is needed")
        return self.d if t.shape[0] < 2 else t.stride(0)

    def reserve_backward(self):
        """Makes the backward's workspace (partial sums of the weight's and bias's gradients) now."""
        ws = self._ws.get("backward")
        if ws is None:
            require(not torch.cuda.is_current_stream_capturing(),
                    "reserve the workspace before the capture (reserve_backward)")
            t = self.dtype  # its size does not grow past some rows
            # of two host threads that come first, both take one's
            ws = self._ws.setdefault("backward", Workspace(B.waste_norm_workspace(self._config(t, t), 1 << 30), self.device))
        return ws

    def forward(self, x, y=None, mean=None, rstd=None, stream=None):
        """y [T, d] (fp32, bf16 or fp16; made as x if None) from x [T, d] of any of these types; rows may be strided.
        mean, rstd [T] fp32 receive what backward needs (both or neither).  y may be x."""
        index = self.index
        if B.device_now() != index:
            with torch.cuda.device(index):
                return self.forward(x, y, mean, rstd, stream)
        ld = self._rows(x, "x")
        T = x.shape[0]
        if y is None:
            y = make((T, self.d), x.dtype, self.device, stream)
        ldy = self._rows(y, "y", T)
        for t, n in ((mean, "mean"), (rstd, "rstd")):
            if t is not None:
                check(t, n, (T,), _F32, self.device)
        B.waste_norm_forward(self._config(x.dtype, y.dtype), x, ld, T, self.weight, self.bias, y, ldy, mean, rstd,
                             B.stream_on(index, stream))
        return y

    def backward(self, dy, x, mean, rstd, dx=None, dw=None, db=None, accumulate: bool = False, stream=None):
        """Gradients for dy [T, d] (of y's type), given forward's x, mean and rstd: into dx [T, d] (x's type), dw and
        db [d] (fp32 or the weight's type), each of them None where it is not wanted; dw and db are added to what is
        there with accumulate.  dx may be dy."""
        index = self.index
        if B.device_now() != index:
            with torch.cuda.device(index):
                return self.backward(dy, x, mean, rstd, dx, dw, db, accumulate, stream)
        ldx = self._rows(x, "x")
        T = x.shape[0]
        lddy = self._rows(dy, "dy", T)
        lddx = 0
        if dx is not None:
            lddx = self._rows(dx, "dx", T)
            if dx.dtype != x.dtype:
                require(False, f"dx: {x.dtype}, as x, is needed")
        check(mean, "mean", (T,), _F32, self.device)
        check(rstd, "rstd", (T,), _F32, self.device)
        gt = (dw if dw is not None else db if db is not None else self.weight).dtype
        for t, n in ((dw, "dw"), (db, "db")):
            if t is not None:
                check(t, n, (self.d,), (gt,) if gt in (self.dtype, torch.float32) else (self.dtype, torch.float32), self.device)
        h = B.stream_on(index, stream)
        args = (self._config(x.dtype, dy.dtype), dy, lddy, x, ldx, T, mean, rstd, self.weight, dx, lddx, dw, db, ACT[gt],
                int(accumulate))
        if dw is None and db is None:
            B.waste_norm_backward(*args, None, h)
            return
        ws = self._ws.get("backward") or self.reserve_backward()
        with ws.one:
            B.waste_norm_backward(*args, ws.lend(stream, h), h)

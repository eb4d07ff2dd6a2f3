"""Updates made orthogonal by Newton-Schulz products (include/waste_train.h: waste_ortho_update), as the Muon optimiser
makes them of a matrix's gradient or momentum.  All computation is in the library's kernels.
"""
from __future__ import annotations

import torch

from . import binding as B
from .dense import ACT, Workspace, check, make, require

_FLOATS = (torch.float32, torch.bfloat16, torch.float16)


class NewtonSchulz:
    """For stacks of `count` matrices [rows, cols]: X = G / |G|, then `steps` times X <- a X + (b A + c A^2) X with
    A = X X^T on the short side; coefficients are a, b and c.  The workspace belongs to this object, which is not made
    during a capture: calls of one object must not run at the same time on two streams (from several host threads on one
    stream they may), two captured graphs that may replay at the same time need an object each, and an object outlives
    the graphs that hold its calls.  stream: a torch.cuda.Stream, an integer handle (then the object must outlive the
    call) or None for the current stream; ordering the tensors' use between streams is the caller's."""

    def __init__(self, count: int, rows: int, cols: int, steps: int = 5, coefficients=(3.4445, -4.7750, 2.0315), device="cuda"):
        dev = torch.device(device)
        require(dev.type == "cuda", "the device is a GPU")
        if dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        require(len(coefficients) == 3, "coefficients are a, b and c")
        self.count, self.rows, self.cols, self.steps = int(count), int(rows), int(cols), int(steps)
        self.coefficients, self.device, self.index = tuple(map(float, coefficients)), dev, dev.index
        self.cfg = B.waste_ortho_config(B.ABI_VERSION, self.count, self.rows, self.cols, self.steps, *self.coefficients)
        need = B.waste_ortho_workspace(self.cfg)
        require(not torch.cuda.is_current_stream_capturing(), "make the object, and its workspace with it, before the capture")
        self._ws = Workspace(need, dev)

    def orthogonalize(self, g, out=None, scale: float = 1.0, mode: int = 0, stream=None):
        """out [count, rows, cols] = (mode 0; bf16, made if None) or += (mode 1; fp32, bf16 or fp16: a weight and its
        update) scale times the orthogonalised g [count, rows, cols] (fp32, bf16 or fp16).  Five steps are off the exact
        update by 1e-3 of its norm or so (16-bit products), onto fp32 weights too.  A stack of one may be given as
        [rows, cols]."""
        index = self.index
        if B.device_now() != index:
            with torch.cuda.device(index):
                return self.orthogonalize(g, out, scale, mode, stream)
        shape = (self.count, self.rows, self.cols)
        if self.count == 1 and isinstance(g, torch.Tensor) and g.dim() == 2:
            shape = shape[1:]
        check(g, "g", shape, _FLOATS, self.device)
        if out is None:
            require(mode == 0, "mode 1 adds to a given out")
            out = make(shape, torch.bfloat16, self.device, stream)
        check(out, "out", shape, _FLOATS if mode else (torch.bfloat16,), self.device)
        h = B.stream_on(index, stream)
        ws = self._ws
        with ws.one:
            B.waste_ortho_update(self.cfg, g, ACT[g.dtype], out, ACT[out.dtype], scale, mode, ws.lend(stream, h), h)
        return out

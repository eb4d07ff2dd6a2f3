"""Microscaled 4-bit matrices (MXFP4), their product, and a dense expert whose weights are held
in them (include/waste_dense.h: waste_mx4_*).

Beside the 3-bit codes of the routed experts (``waste_rvq_train``) this is the cheap format: no
codebooks and no training, a matrix is quantised in one pass, and the tensor core multiplies it
without decoding.  All computation is in the library's kernels.
"""
from __future__ import annotations

import torch

from . import binding as B
from .dense import ACT, Workspace, check, make, require

_FLOATS = (torch.float32, torch.bfloat16, torch.float16)


class Mx4Matrix:
    """codes [rows, cols / 2] uint8 and the scale tiles (uint8, waste_mx4_layout) of a matrix."""

    def __init__(self, rows: int, cols: int, codes: torch.Tensor, scales: torch.Tensor):
        nc, ns = B.waste_mx4_layout(rows, cols)
        dev = codes.device
        require(dev.type == "cuda", "codes and scales are tensors on a GPU")
        check(codes, "codes", (rows, cols // 2), (torch.uint8,), dev)
        check(scales, "scales", (ns,), (torch.uint8,), dev)
        self.rows, self.cols, self.codes, self.scales = rows, cols, codes, scales
        self.device, self.index = dev, dev.index

    @classmethod
    def empty(cls, rows: int, cols: int, device="cuda") -> "Mx4Matrix":
        _, ns = B.waste_mx4_layout(rows, cols)
        return cls(rows, cols, torch.empty(rows, cols // 2, dtype=torch.uint8, device=device),
                   torch.empty(ns, dtype=torch.uint8, device=device))

    @classmethod
    def from_dense(cls, x: torch.Tensor, stream=None) -> "Mx4Matrix":
        require(isinstance(x, torch.Tensor) and x.dim() == 2, "x: a [rows, cols] tensor is needed")
        with torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream) else None):
            m = cls.empty(*x.shape, device=x.device)
        m.quantize(x, stream)
        return m

    def _plain(self, t, name, dtypes=_FLOATS) -> int:
        """The row stride of a [rows, cols] tensor whose rows are contiguous."""
        if not (isinstance(t, torch.Tensor) and t.shape == (self.rows, self.cols) and t.dtype in dtypes
                and t.device == self.device and (self.rows == 0 or t.stride(1) == 1)):
            require(False, f"{name}: a [{self.rows}, {self.cols}] tensor with contiguous rows, fp32, bf16 or fp16, "
                           f"on {self.device} is needed")
        return self.cols if self.rows < 2 else t.stride(0)

    def quantize(self, x: torch.Tensor, stream=None):
        """Replace this matrix by the quantised x [rows, cols]."""
        index = self.index
        if B.device_now() != index:
            with torch.cuda.device(index):
                return self.quantize(x, stream)
        ld = self._plain(x, "x")
        B.waste_mx4_quantize(x, ACT[x.dtype], self.rows, self.cols, ld, self.codes, self.scales,
                             B.stream_on(index, stream))

    def dequantize(self, out: torch.Tensor | None = None, dtype=torch.float32, stream=None) -> torch.Tensor:
        """The values the codes stand for, into out [rows, cols] (made with dtype if None)."""
        index = self.index
        if B.device_now() != index:
            with torch.cuda.device(index):
                return self.dequantize(out, dtype, stream)
        if out is None:
            out = make((self.rows, self.cols), dtype, self.device, stream)
        ld = self._plain(out, "out")
        B.waste_mx4_dequantize(self.codes, self.scales, self.rows, self.cols, out, ACT[out.dtype], ld,
                               B.stream_on(index, stream))
        return out


def matmul(a: Mx4Matrix, b: Mx4Matrix, out: torch.Tensor | None = None, mode: int = 0, dtype=torch.float32,
           stream=None) -> torch.Tensor:
    """out [a.rows, b.rows] (fp32, bf16 or fp16; made with dtype if None) = (mode 0) or += (mode 1)
    a b^T, summed in fp32."""
    if a.cols != b.cols:
        require(False, f"a has {a.cols} columns, b {b.cols}")
    index = a.index
    if b.index != index:
        require(False, "a and b are on two devices")
    if B.device_now() != index:
        with torch.cuda.device(index):
            return matmul(a, b, out, mode, dtype, stream)
    if out is None:
        require(mode == 0, "mode 1 adds to a given out")
        out = make((a.rows, b.rows), dtype, a.device, stream)
    check(out, "out", (a.rows, b.rows), _FLOATS, a.device)
    B.waste_mx4_matmul(a.rows, b.rows, a.cols, a.codes, a.scales, b.codes, b.scales, out, ACT[out.dtype], mode,
                       B.stream_on(index, stream))
    return out


class Mx4Expert:
    """A dense expert with 4-bit weights: gate, up [f, d] and down [d, f] (kept, not copied).
    max_tokens bounds T and sizes the workspace, which belongs to this object: calls of one
    object must not run at the same time on two streams, two captured graphs that may replay at the
    same time need an object each, and an object outlives the graphs that hold its calls.  stream
    and host threads as for ``dense.DenseExpert``."""

    def __init__(self, gate: Mx4Matrix, up: Mx4Matrix, down: Mx4Matrix, max_tokens: int):
        f, d = gate.rows, gate.cols
        require((up.rows, up.cols) == (f, d) and (down.rows, down.cols) == (d, f),
                "gate and up are [f, d], down is [d, f]")
        require(gate.device == up.device == down.device, "the matrices are on two devices")
        require(max_tokens >= 1, "max_tokens >= 1")
        self.gate, self.up, self.down = gate, up, down
        self.d, self.f, self.device, self.index, self.max_tokens = d, f, gate.device, gate.index, int(max_tokens)
        self.cfg = B.waste_mx4_ffn_config(B.ABI_VERSION, d, f, *(t.data_ptr() for m in (gate, up, down)
                                                                 for t in (m.codes, m.scales)))
        self._ws = Workspace(B.waste_mx4_ffn_workspace(self.cfg, self.max_tokens), self.device)

    @classmethod
    def from_dense(cls, w_gate, w_up, w_down, max_tokens: int) -> "Mx4Expert":
        return cls(*(Mx4Matrix.from_dense(w) for w in (w_gate, w_up, w_down)), max_tokens=max_tokens)

    def forward(self, x, out=None, mode: int = 0, stream=None):
        """out [T, d] (fp32, bf16 or fp16; made as x if None) = (mode 0) or += (mode 1) the block's
        output for x [T, d].  out may be x."""
        index = self.index
        if B.device_now() != index:
            with torch.cuda.device(index):
                return self.forward(x, out, mode, stream)
        require(isinstance(x, torch.Tensor) and x.dim() == 2, "x: a [T, d] tensor is needed")
        T = x.shape[0]
        if T > self.max_tokens:
            require(False, f"T = {T} exceeds max_tokens = {self.max_tokens}")
        check(x, "x", (T, self.d), _FLOATS, self.device)
        if out is None:
            require(mode == 0, "mode 1 adds to a given out")
            out = make((T, self.d), x.dtype, self.device, stream)
        check(out, "out", (T, self.d), _FLOATS, self.device)
        h = B.stream_on(index, stream)
        ws = self._ws
        with ws.one:
            B.waste_mx4_ffn_forward(self.cfg, x, ACT[x.dtype], T, out, ACT[out.dtype], mode, ws.lend(stream, h), h)
        return out

"""A dense expert: the gated feed-forward block of the routed experts on 16-bit weights, forward
and backward (include/waste_dense.h: waste_ffn_forward, waste_ffn_backward).

Models put such an expert beside the routed ones, applied to every token; an expert is also
trained in this form before its matrices are encoded (``waste_rvq_train``).  All computation
is in the library's kernels.
"""
from __future__ import annotations

import threading

import torch

from . import binding as B

ACT = {torch.float32: B.ACT_F32, torch.bfloat16: B.ACT_BF16, torch.float16: B.ACT_F16}


def require(ok: bool, message: str):
    if not ok:
        raise B.WasteError(-1, message)


def check(t, name: str, shape, dtypes, device):
    """A contiguous tensor of the given shape, on the given device, of one of the types."""
    if not (isinstance(t, torch.Tensor) and t.shape == shape and t.dtype in dtypes and t.device == device
            and t.is_contiguous()):
        require(False, f"{name}: a contiguous tensor of shape {tuple(shape)} and type "
                       f"{' or '.join(map(str, dtypes))} on {device} is needed")


def make(shape, dtype, device, stream) -> torch.Tensor:
    """An output made for a call on `stream` (None or an integer handle: made on the current one)."""
    with torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream) else None):
        return torch.empty(shape, dtype=dtype, device=device)


class Workspace:
    """A buffer made on one stream and lent to calls on any: the allocator is told of the others, so
    that its memory is not given away while a call there still runs.  one: held while a call is
    enqueued, so that the launches of two host threads' calls do not mix."""

    def __init__(self, nbytes: int, device):
        self.bytes = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
        self.home = B.stream_on(device.index, None)
        self.one = threading.Lock()

    def __getstate__(self):
        return self.bytes, self.home

    def __setstate__(self, state):
        self.bytes, self.home = state
        self.one = threading.Lock()

    def lend(self, stream, handle: int) -> torch.Tensor:
        """For a call on `stream`, whose handle is given."""
        if handle != self.home and not isinstance(stream, int):
            self.bytes.record_stream(torch.cuda.current_stream(self.bytes.device) if stream is None else stream)
        return self.bytes


class DenseExpert:
    """w_gate, w_up [f, d] and w_down [d, f], bf16 or fp16, contiguous on one GPU (borrowed, not
    copied).  max_tokens bounds T and sizes the workspace, which belongs to this object: calls
    of one object must not run at the same time on two streams (from several host threads on one
    stream they may: a lock keeps a call's launches together), two captured graphs that may
    replay at the same time need an object each, and an object outlives the graphs that hold its
    calls.  A device wait that gave up shows in ``binding.waste_dense_status``.  stream: a torch.cuda.Stream, an integer handle (then the object must outlive the
    call) or None for the current stream; ordering the tensors' use between streams is the
    caller's."""

    def __init__(self, w_gate: torch.Tensor, w_up: torch.Tensor, w_down: torch.Tensor, max_tokens: int):
        f, d = w_gate.shape
        dev, t = w_gate.device, w_gate.dtype
        require(dev.type == "cuda" and dev.index is not None and t in (torch.bfloat16, torch.float16),
                "weights are bf16 or fp16 tensors on a GPU")
        check(w_gate, "w_gate", (f, d), (t,), dev)
        check(w_up, "w_up", (f, d), (t,), dev)
        check(w_down, "w_down", (d, f), (t,), dev)
        require(max_tokens >= 1, "max_tokens >= 1")
        self.w_gate, self.w_up, self.w_down = w_gate, w_up, w_down
        self.d, self.f, self.dtype, self.device, self.index, self.max_tokens = d, f, t, dev, dev.index, int(max_tokens)
        self._own, self._out = (t,), (t, torch.float32)  # types of inputs, and of outputs
        self.cfg = B.waste_ffn_config(B.ABI_VERSION, d, f, ACT[t])
        self._ws = {}
        self._workspace(0)

    def _workspace(self, backward: int) -> Workspace:
        """One workspace for the forward and one, made by the first call, for the backward; a call
        that would make it while its stream is being captured is refused (the buffer would
        belong to the graph)."""
        ws = self._ws.get(backward)
        if ws is None:
            require(not torch.cuda.is_current_stream_capturing(),
                    "reserve the workspace before the capture (reserve_backward)")
            # of two host threads that come first, both take one's
            ws = self._ws.setdefault(backward, Workspace(B.waste_ffn_workspace(self.cfg, self.max_tokens, backward),
                                                         self.device))
        return ws

    def reserve_backward(self):
        """Makes the backward's workspace (three [max_tokens, f] buffers, and partial sums of few tokens) now."""
        self._workspace(1)

    def _tokens(self, x, name):
        if not isinstance(x, torch.Tensor) or x.dim() != 2:
            require(False, f"{name}: a [T, d] tensor is needed")
        T = x.shape[0]
        if T > self.max_tokens:
            require(False, f"T = {T} exceeds max_tokens = {self.max_tokens}")
        check(x, name, (T, self.d), self._own, self.device)
        return T

    def forward(self, x, out=None, mode: int = 0, save_g=None, save_u=None, stream=None):
        """out [T, d] (fp32 or the weights' type; made if None) = (mode 0) or += (mode 1) the
        block's output for x [T, d].  save_g, save_u [T, f] receive what backward needs.  out may be
        x; nothing else that is written may overlap anything of the call."""
        index = self.index
        if B.device_now() != index:
            with torch.cuda.device(index):
                return self.forward(x, out, mode, save_g, save_u, stream)
        T = self._tokens(x, "x")
        if out is None:
            require(mode == 0, "mode 1 adds to a given out")
            out = make((T, self.d), self.dtype, self.device, stream)
        check(out, "out", (T, self.d), self._out, self.device)
        for t, n in ((save_g, "save_g"), (save_u, "save_u")):
            if t is not None:
                check(t, n, (T, self.f), self._own, self.device)
        h = B.stream_on(index, stream)
        ws = self._ws[0]
        with ws.one:
            B.waste_ffn_forward(self.cfg, x, T, self.w_gate, self.w_up, self.w_down, out, ACT[out.dtype], mode, save_g,
                                save_u, ws.lend(stream, h), h)
        return out

    def backward(self, dy, x, g, u, dx=None, dw_gate=None, dw_up=None, dw_down=None, accumulate: bool = False,
                 stream=None):
        """Gradients for dy [T, d], given forward's x, g and u: into dx [T, d] (None: not computed)
        and the three weights' gradients (all or none; fp32 or the weights' type), added to
        what is there with accumulate.  No output may overlap anything else of the call (dx
        over dy, say): refused."""
        index = self.index
        if B.device_now() != index:
            with torch.cuda.device(index):
                return self.backward(dy, x, g, u, dx, dw_gate, dw_up, dw_down, accumulate, stream)
        T = self._tokens(dy, "dy")
        check(x, "x", (T, self.d), self._own, self.device)
        check(g, "g", (T, self.f), self._own, self.device)
        check(u, "u", (T, self.f), self._own, self.device)
        if dx is not None:
            check(dx, "dx", (T, self.d), self._own, self.device)
        gt = self.dtype if dw_gate is None else dw_gate.dtype
        for t, n, w in ((dw_gate, "dw_gate", self.w_gate), (dw_up, "dw_up", self.w_up),
                        (dw_down, "dw_down", self.w_down)):
            if t is not None:
                check(t, n, w.shape, (gt,) if gt in self._out else self._out, self.device)
        h = B.stream_on(index, stream)
        ws = self._workspace(1)
        with ws.one:
            B.waste_ffn_backward(self.cfg, dy, T, x, g, u, self.w_gate, self.w_up, self.w_down, dx, dw_gate, dw_up,
                                 dw_down, ACT[gt], int(accumulate), ws.lend(stream, h), h)

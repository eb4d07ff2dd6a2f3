"""How the dense operators may be called: on memory that overlaps, with sizes past 32 bits, right behind
what writes their weights, first in a process, from several host threads, in decode stacks of every kind, on copies
of an expert."""
import copy
import os
import pickle
import subprocess
import sys
import threading

import pytest
import torch

from rvq_compressed_expert_gb300 import binding as B
from rvq_compressed_expert_gb300 import synth
from rvq_compressed_expert_gb300.bank import TieredStack
from rvq_compressed_expert_gb300.dense import DenseExpert
from rvq_compressed_expert_gb300.layer import MoELayer
from rvq_compressed_expert_gb300.mx4 import Mx4Expert, Mx4Matrix, matmul
from rvq_compressed_expert_gb300.stack import DecodeStack

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from rvq_compressed_expert_gb300 import _build
    _build.build()
    B.load()


def gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def randn(g, *shape, scale=1.0, t=FP):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(t)


def weights(g, d, f, t):
    return randn(g, f, d, scale=d ** -0.5, t=t), randn(g, f, d, scale=d ** -0.5, t=t), randn(g, d, f, scale=f ** -0.5, t=t)


# ---------------------------------------------------------------- overlapping memory

@pytest.mark.parametrize("T,d,f", [(1, 2048, 264), (2, 2048, 264), (7, 1032, 136), (32, 4104, 520), (64, 1032, 264), (131, 2056, 520),
                                   (300, 520, 264), (1000, 1032, 392)])
def test_forward_in_place(T, d, f):
    """out = x, and x += block(x): the bits of a call with memory of its own."""
    g = gen(T + d)
    e = DenseExpert(*weights(g, d, f, BF), max_tokens=T)
    x = randn(g, T, d, t=BF)
    want = e.forward(x)
    added = e.forward(x, x.clone(), mode=1)
    for mode, ref in ((0, want), (1, added)):
        y = x.clone()
        e.forward(y, y, mode=mode)
        assert torch.equal(y, ref)
    d, f = d // 32 * 32, f // 32 * 32
    q = Mx4Expert.from_dense(*weights(g, d, f, BF), max_tokens=T)
    x = randn(g, T, d)
    want, added = q.forward(x), q.forward(x, x.clone(), mode=1)
    for mode, ref in ((0, want), (1, added)):
        y = x.clone()
        q.forward(y, y, mode=mode)
        assert torch.equal(y, ref)


def test_overlaps_are_refused():
    g = gen(1)
    T, d, f = 20, 64, 32
    W = weights(g, d, f, BF)
    e = DenseExpert(*W, max_tokens=T)
    x, dy, sg, su = (randn(g, T, n, t=BF) for n in (d, d, f, f))
    dw = [torch.empty_like(w) for w in W]
    keep = [v.clone() for v in (x, dy, sg, su, *W)]
    both = torch.empty(2 * f, d, dtype=BF, device="cuda")
    for call in (lambda: e.backward(dy, x, sg, su, dy, *dw), lambda: e.backward(dy, x, sg, su, x, *dw),
                 lambda: e.backward(dy, x, sg, su, None, W[0], *dw[1:]),
                 lambda: e.backward(dy, x, sg, su, None, both[:f], both[8:f + 8], dw[2]),
                 lambda: e.forward(x, save_g=sg, save_u=sg), lambda: e.forward(x, W[0].view(-1)[:T * d].view(T, d))):
        with pytest.raises(B.WasteError) as ei:
            call()
        assert ei.value.status == -1
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(keep, (x, dy, sg, su, *W)))
    # inputs may be one tensor, gradients neighbours in one buffer
    dx = torch.empty_like(x)
    e.backward(dy, dy, sg, sg, dx, both[:f], both[f:], dw[2])
    dw2 = [torch.empty_like(w) for w in W]
    e.backward(dy, dy.clone(), sg, sg.clone(), None, *dw2)
    assert torch.equal(both[:f], dw2[0]) and torch.equal(both[f:], dw2[1]) and torch.equal(dw[2], dw2[2])


def test_codes_between_strided_rows():
    """Codes and scales in the gaps between x's rows (and then out's) overlap nothing."""
    rows, cols, ld = 5, 96, 512
    g = gen(2)
    buf = torch.zeros(rows + 1, ld, device="cuda")
    x = buf[:rows, :cols]
    x.copy_(randn(g, rows, cols))
    want = Mx4Matrix.from_dense(x.clone())
    codes, scales = buf[0, cols:cols + rows * cols // 8], buf[1, cols:cols + want.scales.numel() // 4]
    values = x.clone()
    B.waste_mx4_quantize(x, B.ACT_F32, rows, cols, ld, codes, scales)
    assert torch.equal(codes.view(torch.uint8), want.codes.view(-1)) and torch.equal(scales.view(torch.uint8), want.scales)
    assert torch.equal(x, values)
    B.waste_mx4_dequantize(codes, scales, rows, cols, x, B.ACT_F32, ld)
    assert torch.equal(x, want.dequantize())


# ---------------------------------------------------------------- sizes past 2^30

def test_sizes_past_32_bits_are_refused():
    """Sizes that are other, small ones in 32 bits (one token, f = 8, one row tile): refused, not taken for those."""
    W = weights(gen(3), 64, 32, BF)
    far = 1 << 32
    q = [Mx4Matrix.from_dense(w) for w in W]
    for n in (far + 1, far + 300, (1 << 30) + 1):
        for make in (lambda: DenseExpert(*W, max_tokens=n), lambda: Mx4Expert(*q, max_tokens=n)):
            with pytest.raises(B.WasteError) as ei:
                make()
            assert ei.value.status == -1
    room = torch.empty(8 * (far + 32), dtype=BF, device="cuda")  # 69 GB, not touched
    w = codes = None
    try:
        w = room.view(far + 32, 8)
        with pytest.raises(B.WasteError):
            DenseExpert(w, w, room.view(8, far + 32), max_tokens=1)
        with pytest.raises(B.WasteError):
            DenseExpert(room.view(8, far + 32), room.view(8, far + 32), w, max_tokens=1)
        codes = room.view(torch.uint8)[:(far + 32) * 16].view(far + 32, 16)
        with pytest.raises(B.WasteError):
            Mx4Matrix(far + 32, 32, codes, torch.empty(512, dtype=torch.uint8, device="cuda"))
        with pytest.raises(B.WasteError):
            Mx4Matrix(1, far + 32, codes.view(-1)[:(far + 32) // 2].view(1, -1), torch.empty(512, dtype=torch.uint8, device="cuda"))
    finally:
        del room, w, codes
        torch.cuda.empty_cache()


# ---------------------------------------------------------------- what stands right before a call

@pytest.mark.parametrize("T", [1, 2, 3, 20, 64, 131, 600])
def test_weights_written_just_before(T):
    """Weights that the operators' own kernels write right before the calls that read them, the down matrix last (its
    first rows are asked for ahead of a wait): each call sees the newest."""
    d, f, n = 2048, 768, 40
    g = gen(T)
    sets = [weights(g, d, f, FP) for _ in range(2)]
    fours = [[Mx4Matrix.from_dense(w) for w in ws] for ws in sets]
    x, dy, sg, su = (randn(g, T, k, t=BF) for k in (d, d, f, f))
    W = [torch.empty_like(w, dtype=BF) for w in sets[0]]
    e = DenseExpert(*W, max_tokens=T)
    m = [Mx4Matrix.empty(*w.shape) for w in W]
    q = Mx4Expert(*m, max_tokens=T)
    want = []
    for four in fours:
        for a, w in zip(four, W):
            a.dequantize(w)
        torch.cuda.synchronize()
        y, dx = e.forward(x), torch.empty_like(x)
        e.backward(dy, x, sg, su, dx)
        want.append((y, dx, Mx4Expert(*four, max_tokens=T).forward(x)))
        torch.cuda.synchronize()
    assert not any(torch.equal(a, b) for a, b in zip(*want))
    got = [[torch.empty_like(x) for _ in range(3)] for _ in range(n)]
    for i, (y, dx, y4) in enumerate(got):
        for a, w in zip(fours[i & 1], W):
            a.dequantize(w)
        e.forward(x, y)
        fours[1 - (i & 1)][1].dequantize(W[1])  # and the order of the backward's
        for j in (2, 0, 1):
            fours[i & 1][j].dequantize(W[j])
        e.backward(dy, x, sg, su, dx)
        for a, w in zip(m, sets[i & 1]):
            a.quantize(w)
        q.forward(x, y4)
    torch.cuda.synchronize()
    for i, out in enumerate(got):
        assert all(torch.equal(a, b) for a, b in zip(out, want[i & 1])), i


@pytest.mark.parametrize("T", [1, 3, 40, 300])
def test_captured_behind_memsets_copies_and_joins(T):
    """Calls recorded right behind a memset, a copy, and the join of two streams (nodes that are no kernels, or several
    of them), and calls with such nodes behind them: the replay gives eager bits."""
    d, f = 512, 256
    g = gen(T)
    W = weights(g, d, f, BF)
    e, q = DenseExpert(*W, max_tokens=T), Mx4Expert.from_dense(*W, max_tokens=T)
    e.reserve_backward()
    src, x, x2, dy, sg, su = (randn(g, T, n, t=BF) for n in (d, d, d, d, f, f))
    y, y4, dx, back = (torch.empty(T, d, dtype=BF, device="cuda") for _ in range(4))
    dw, m, c = [torch.empty_like(w) for w in W], Mx4Matrix.empty(T, d), torch.empty(T, f, device="cuda")
    side = torch.cuda.Stream()
    now = torch.cuda.current_stream

    def calls():
        for v in (y, y4, dx):
            v.zero_()
        x.copy_(src)                       # a copy, then the call that reads it
        e.forward(x, y, mode=1)
        side.wait_stream(now())
        with torch.cuda.stream(side):
            x2.copy_(y)                    # a copy behind a call
            q.forward(x2, y4, mode=1)
        c.zero_()
        m.quantize(x)
        matmul(m, q.gate, c, mode=1)
        now().wait_stream(side)             # two predecessors
        e.backward(dy, y4, sg, su, dx, *dw)
        dy.copy_(dx)
        e.backward(dy, x, sg, su, dx, *dw, accumulate=True)
        back.copy_(dx)
        m.dequantize(dx)

    out = [y, y4, dx, back, c, *dw]
    keep = dy.clone()
    warm = torch.cuda.Stream()
    warm.wait_stream(now())
    with torch.cuda.stream(warm):
        calls()
    torch.cuda.synchronize()
    want = [v.clone() for v in out]
    dy.copy_(keep)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        calls()
    for _ in range(3):
        dy.copy_(keep)
        for v in out:
            v.fill_(float("nan"))
        gr.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    assert all(torch.isfinite(v.float()).all() for v in want)


FIRST = """
import sys, torch
from rvq_compressed_expert_gb300 import binding as B
from rvq_compressed_expert_gb300.dense import DenseExpert
from rvq_compressed_expert_gb300.mx4 import Mx4Expert, Mx4Matrix, matmul
T, d, f = int(sys.argv[1]), 512, 256
torch.manual_seed(1)
rn = lambda *s: torch.randn(*s, device="cuda").bfloat16()
W = [rn(f, d) / 20, rn(f, d) / 20, rn(d, f) / 16]
x, dy, g, u = rn(T, d), rn(T, d), rn(T, f), rn(T, f)
e, m, M4 = DenseExpert(*W, max_tokens=T), Mx4Matrix.empty(T, d), [Mx4Matrix.empty(*w.shape) for w in W]
e.reserve_backward()
q = Mx4Expert(*M4, max_tokens=T)
out = [torch.empty_like(x) for _ in range(3)] + [torch.empty_like(w) for w in W] + [torch.empty(T, f, device="cuda"), x.float()]
def calls():
    e.forward(x, out[0])
    e.backward(dy, x, g, u, out[1], *out[3:6])
    m.quantize(x)
    for a, b in zip(M4, W):
        a.quantize(b)
    matmul(m, M4[0], out[6])
    q.forward(x, out[2])
    m.dequantize(out[7])
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    calls()
graph.replay()
torch.cuda.synchronize()
first = [o.clone() for o in out]
calls()
torch.cuda.synchronize()
B.waste_dense_status()
assert all(torch.equal(a, b) and torch.isfinite(a.float()).all() for a, b in zip(first, out))
print("same")
"""


@pytest.mark.parametrize("T", [1, 20, 300])
def test_first_calls_of_a_process_are_captured(T):
    """A process whose first calls of every operator are recorded into a graph: its replay gives an eager call's bits."""
    r = subprocess.run([sys.executable, "-c", FIRST, str(T)], capture_output=True, text=True, timeout=120,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr[-2000:]


# ---------------------------------------------------------------- several host threads

def in_threads(*work):
    """Every function in a thread of its own, begun together; the first error is raised here."""
    gate, errors = threading.Barrier(len(work)), []

    def run(f):
        try:
            gate.wait()
            f()
        except BaseException as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run, args=(f,)) for f in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if errors:
        raise errors[0]


@pytest.mark.parametrize("T", [1, 2, 20, 150, 600])
def test_first_calls_of_a_thread(T):
    """A host thread whose first use of CUDA is a call of these operators (no context is current in it yet)."""
    d, f = 320, 160
    g = gen(T)
    W = weights(g, d, f, BF)
    e, q = DenseExpert(*W, max_tokens=T), Mx4Expert.from_dense(*W, max_tokens=T)
    e.reserve_backward()
    x, dy, sg, su = (randn(g, T, n, t=BF) for n in (d, d, f, f))
    a, s = Mx4Matrix.from_dense(x), torch.cuda.Stream()
    y, dx, y4, back = (torch.empty_like(x) for _ in range(4))
    dw, c = [torch.empty_like(w) for w in W], torch.empty(T, f, device="cuda")
    m = Mx4Matrix.empty(T, d)
    calls = {"forward": (lambda: e.forward(x, y, stream=s), [y]), "backward": (lambda: e.backward(dy, x, sg, su, dx, *dw, stream=s), [dx, *dw]),
             "quantize": (lambda: m.quantize(x, stream=s), [m.codes, m.scales]), "dequantize": (lambda: a.dequantize(back, stream=s), [back]),
             "matmul": (lambda: matmul(a, q.gate, c, stream=s), [c]), "block": (lambda: q.forward(x, y4, stream=s), [y4])}
    for name, (call, out) in calls.items():
        call()
        torch.cuda.synchronize()
        want = [v.clone() for v in out]
        for v in out:
            v.zero_()
        torch.cuda.synchronize()
        in_threads(call)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), name


@pytest.mark.parametrize("T,d,f", [(3, 1032, 264), (40, 1032, 264), (150, 520, 392)])
def test_one_expert_in_two_threads(T, d, f):
    """Calls of one object from two host threads on one stream, the first backward (which makes its workspace)
    among them: each thread gets the bits of its own inputs."""
    g = gen(T)
    W = weights(g, d, f, BF)
    sets = [[randn(g, T, n, t=BF) for n in (d, d, f, f)] for _ in range(2)]
    alone = DenseExpert(*W, max_tokens=T)
    q = Mx4Expert.from_dense(*(w[:, : w.shape[1] // 32 * 32][: w.shape[0] // 32 * 32].contiguous() for w in W), max_tokens=T)
    xq = [s[0][:, :q.d].contiguous() for s in sets]
    want = []
    for s, xs in zip(sets, xq):
        out = [torch.empty(T, d, dtype=BF, device="cuda") for _ in range(2)] + [torch.empty_like(w) for w in W]
        alone.forward(s[0], out[0])
        alone.backward(*s, *out[1:])
        want.append(out + [q.forward(xs)])
    torch.cuda.synchronize()
    for again in range(3):
        e = DenseExpert(*W, max_tokens=T)
        n = 150
        got = [[[torch.empty_like(v) for v in w] for _ in range(n)] for w in want]
        torch.cuda.synchronize()

        def calls(i):
            def run():
                for out in got[i]:
                    e.backward(*sets[i], *out[1:5])
                    e.forward(sets[i][0], out[0])
                    q.forward(xq[i], out[5])
            return run

        in_threads(calls(0), calls(1))
        torch.cuda.synchronize()
        for i in range(2):
            wrong = sum(not torch.equal(a, b) for out in got[i] for a, b in zip(out, want[i]))
            assert wrong == 0, (again, i, wrong)


def test_two_experts_in_two_threads():
    """Experts of their own on streams of their own, of sizes that need different shared memory of the same kernels."""
    sizes = [(17, 2056, 1032), (170, 520, 136)]
    work, checks = [], []
    for T, d, f in sizes:
        g = gen(T)
        e = DenseExpert(*weights(g, d, f, HF), max_tokens=T)
        x, s = randn(g, T, d, t=HF), torch.cuda.Stream()
        want = e.forward(x).clone()
        outs = [torch.empty_like(want) for _ in range(100)]
        torch.cuda.synchronize()

        def run(e=e, x=x, s=s, outs=outs):
            for out in outs:
                e.forward(x, out, stream=s)

        work.append(run)
        checks.append((want, outs))
    in_threads(*work)
    torch.cuda.synchronize()
    for want, outs in checks:
        assert all(torch.equal(want, o) for o in outs)


# ---------------------------------------------------------------- shared experts of decode stacks

def workload(tokens):
    return synth.Workload("shared-calls", 512, 256, 16, 4, tokens, "f32", "offsets", n_layers=4, lookahead=3)


def shared_experts(tokens):
    g = gen(60)
    return [DenseExpert(*weights(g, 512, 256, BF), max_tokens=tokens), Mx4Expert.from_dense(*weights(g, 512, 160, BF), max_tokens=tokens),
            None, DenseExpert(*weights(g, 512, 264, HF), max_tokens=tokens + 5)]


def eager(stack, hidden, lookahead):
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    main.wait_stream(torch.cuda.current_stream())
    outs = []
    for h in hidden:
        out = stack.run(h, lookahead, main, side)
        with torch.cuda.stream(main):
            outs.append(out.clone())
    torch.cuda.synchronize()
    return outs


@pytest.mark.parametrize("lookahead", [0, 3])
@pytest.mark.parametrize("tokens", [1, 3])
def test_stack_of_shared_experts_captured(tokens, lookahead):
    """A pass through layers with dense (bf16, fp16) and 4-bit shared experts, recorded into a graph and replayed
    on other tokens, gives the bits of eager passes, and each layer's residual is the layer's parts one by one."""
    w = workload(tokens)
    layers = [MoELayer(w, 0, L, "cuda") for L in range(w.n_layers)]
    try:
        shared = shared_experts(tokens)
        stack = DecodeStack(layers, tokens, shared=shared)
        hidden = [synth.hidden(70 + i, tokens, w.d, "f32", "cuda") for i in range(3)]
        want = eager(stack, hidden, lookahead)
        h, x = hidden[0].clone(), torch.empty_like(hidden[0])
        idx, gate, logits, _ = layers[0].alloc_outputs(tokens)
        for L, e in enumerate(shared):
            B.waste_moe_rmsnorm(h, x, tokens, w.d)
            layers[L].route(x, tokens, idx, gate, logits)
            layers[L].forward(x, tokens, idx, gate, h, 1)
            if e is not None:
                e.forward(x.to(e.dtype) if isinstance(e, DenseExpert) else x, h, mode=1)
        torch.cuda.synchronize()
        assert torch.equal(want[0], h)
        h0, main, side = hidden[0].clone(), torch.cuda.Stream(), torch.cuda.Stream()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=main):
            out = stack.run(h0, lookahead, main, side)
        for i in (2, 0, 1):
            h0.copy_(hidden[i])
            gr.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want[i])
        del gr
        B.waste_dense_status()
    finally:
        for m in layers:
            m.close()


@pytest.mark.parametrize("lookahead", [0, 3])
def test_banked_stack_with_shared_experts(lookahead):
    """Layers whose records come through an HBM cache that evicts, with shared experts: the resident stack's bits."""
    w = workload(1)
    hidden = [synth.hidden(80 + i, 1, w.d, "f32", "cuda") for i in range(4)]
    layers = [MoELayer(w, 0, L, "cuda") for L in range(w.n_layers)]
    try:
        want = eager(DecodeStack(layers, 1, shared=shared_experts(1)), hidden, lookahead)
        plain = eager(DecodeStack(layers, 1), hidden, lookahead)
    finally:
        for m in layers:
            m.close()
    ts = TieredStack(w, 0, w.n_layers, 6)
    try:
        got = eager(DecodeStack(ts.layers, 1, banked=True, shared=shared_experts(1)), hidden, lookahead)
        for a, b, c in zip(got, want, plain):
            assert torch.equal(a, b) and not torch.equal(a, c)
        for m in ts.layers:
            m.stats()
    finally:
        ts.close()


# ---------------------------------------------------------------- copies of an expert

def test_copies_of_an_expert():
    """A shallow copy (it shares the workspace, and what keeps two threads' calls apart in it), a deep one and one
    through pickle give the same bits, forward and backward."""
    T, d, f = 40, 64, 32
    g = gen(9)
    e = DenseExpert(*weights(g, d, f, BF), max_tokens=T)
    x, dy, sg, su = (randn(g, T, n, t=BF) for n in (d, d, f, f))
    want, dx = e.forward(x), torch.empty_like(x)
    e.backward(dy, x, sg, su, dx)
    for twin in (copy.copy(e), copy.deepcopy(e), pickle.loads(pickle.dumps(e))):
        got = torch.empty_like(dx)
        twin.backward(dy, x, sg, su, got)
        assert torch.equal(twin.forward(x), want) and torch.equal(got, dx)
        assert (twin._ws[0].one is e._ws[0].one) == (twin._ws[0].bytes.data_ptr() == e._ws[0].bytes.data_ptr())
    q = Mx4Expert.from_dense(*weights(g, d, f, BF), max_tokens=T)
    assert torch.equal(copy.copy(q).forward(x), q.forward(x))

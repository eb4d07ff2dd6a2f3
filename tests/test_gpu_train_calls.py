"""How the training operators may be called: captured and replayed, on other streams and from other host threads, beside
other work, on more than 2^31 elements, in a decode stack, and one behind another as in a training step."""
import copy
import pickle
import threading

import pytest
import torch

from rvq_compressed_expert_gb300 import binding as B
from rvq_compressed_expert_gb300 import synth
from rvq_compressed_expert_gb300.bank import TieredStack
from rvq_compressed_expert_gb300.grouped import GroupedLinear
from rvq_compressed_expert_gb300.layer import MoELayer
from rvq_compressed_expert_gb300.norm import LayerNorm
from rvq_compressed_expert_gb300.ortho import NewtonSchulz
from rvq_compressed_expert_gb300.stack import DecodeStack
from tests import train_ref as R

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from rvq_compressed_expert_gb300 import _build
    _build.build()
    B.load()


@pytest.fixture(autouse=True)
def _status():
    yield
    B.waste_dense_status()


def gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def randn(g, *shape, scale=1.0, t=FP):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(t)


class Calls:
    """Every operator once, on inputs that `fill` changes in place."""

    def __init__(self, T, d, sizes, k, n, count, rows, cols):
        g = gen(T)
        self.sizes, self.E = sizes, len(sizes)
        R_ = sum(sizes)
        self.w, self.b = randn(g, d, t=BF), randn(g, d, t=BF)
        self.x, self.dy = randn(g, T, d, t=BF), randn(g, T, d, t=BF)
        self.gw, self.gx, self.gdy = randn(g, self.E, n, k, t=HF), randn(g, R_, k, t=HF), randn(g, R_, n, t=HF)
        self.off = torch.zeros(self.E + 1, dtype=torch.int32, device="cuda")
        self.G = randn(g, count, rows, cols)
        self.norm, self.grouped, self.ns = LayerNorm(self.w, self.b), GroupedLinear(self.gw), NewtonSchulz(count, rows, cols)
        self.norm.reserve_backward()
        e = torch.empty_like
        f32 = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
        self.out = dict(y=e(self.x), mean=f32(T), rstd=f32(T), dx=e(self.x), dw=f32(d), db=f32(d), gy=torch.empty(R_, n, dtype=HF, device="cuda"),
                        gdx=e(self.gx), gdw=e(self.gw), o=torch.empty(count, rows, cols, dtype=BF, device="cuda"))
        self.fill(0)

    def fill(self, seed):
        g = gen(100 + seed)
        for t in (self.w, self.b, self.x, self.dy, self.gw, self.gx, self.gdy, self.G):
            t.copy_(randn(g, *t.shape))
        order = torch.randperm(self.E, generator=torch.Generator().manual_seed(seed))
        self.off[1:] = torch.tensor(self.sizes)[order].cumsum(0).cuda()
        for t in self.out.values():
            t.fill_(3.0)

    def run(self, stream=None):
        o = self.out
        self.norm.forward(self.x, o["y"], o["mean"], o["rstd"], stream=stream)
        self.norm.backward(self.dy, self.x, o["mean"], o["rstd"], o["dx"], o["dw"], o["db"], stream=stream)
        self.grouped.forward(self.gx, self.off, o["gy"], stream=stream)
        self.grouped.backward(self.gdy, self.gx, self.off, o["gdx"], o["gdw"], stream=stream)
        self.ns.orthogonalize(self.G, o["o"], stream=stream)

    def kept(self):
        torch.cuda.synchronize()
        return {k: v.clone() for k, v in self.out.items()}


SHAPES = [(5, 40, [3, 0, 1, 7], 64, 40, 3, 24, 100), (1500, 1024, [200, 0, 331, 190, 161], 264, 200, 1, 200, 520),
          (700, 2001, [1000], 72, 328, 2, 520, 136)]


def same(a, b):
    return all(torch.equal(a[k].view(torch.uint8) if a[k].dtype == BF else a[k], b[k].view(torch.uint8) if b[k].dtype == BF else b[k]) for k in a)


@pytest.mark.parametrize("shape", SHAPES)
def test_captured_and_replayed(shape):
    """Recorded once, replayed on other inputs and other offsets: the bits of eager calls."""
    c = Calls(*shape)
    want = []
    for i in range(4):
        c.fill(i)
        c.run()
        want.append(c.kept())
    gr = torch.cuda.CUDAGraph()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(gr, stream=s):
        c.run()
    for i in (3, 0, 2, 1):
        c.fill(i)
        gr.replay()
        assert same(c.kept(), want[i])
    del gr


@pytest.mark.parametrize("shape", SHAPES)
def test_streams_and_busy_gpu(shape):
    """On a stream of its own, by handle, and again beside another stream's work: the same bits every time."""
    c = Calls(*shape)
    c.run()
    want = c.kept()
    s, other = torch.cuda.Stream(), torch.cuda.Stream()
    a = torch.randn(2048, 2048, device="cuda")
    torch.cuda.synchronize()
    for how in (s, s.cuda_stream, s, s):
        for t in c.out.values():
            t.fill_(3.0)
        torch.cuda.synchronize()
        with torch.cuda.stream(other):
            for _ in range(20):
                a = torch.tanh(a @ a)
        c.run(how)
        assert same(c.kept(), want)


def test_first_calls_of_a_thread():
    """Each operator as the first thing that a host thread does with CUDA."""
    c = Calls(*SHAPES[1])
    c.run()
    want, failed = c.kept(), []
    h = torch.cuda.Stream().cuda_stream
    for f in ("forward", "backward", "gforward", "gbackward", "ortho"):
        def work():
            try:
                o = c.out
                {"forward": lambda: c.norm.forward(c.x, o["y"], o["mean"], o["rstd"], stream=h),
                 "backward": lambda: c.norm.backward(c.dy, c.x, o["mean"], o["rstd"], o["dx"], o["dw"], o["db"], stream=h),
                 "gforward": lambda: c.grouped.forward(c.gx, c.off, o["gy"], stream=h),
                 "gbackward": lambda: c.grouped.backward(c.gdy, c.gx, c.off, o["gdx"], o["gdw"], stream=h),
                 "ortho": lambda: c.ns.orthogonalize(c.G, o["o"], stream=h)}[f]()
            except Exception as e:  # noqa: BLE001
                failed.append((f, e))
        t = threading.Thread(target=work)
        t.start()
        t.join()
        torch.cuda.synchronize()
    assert not failed and same(c.kept(), want)


def test_one_object_in_two_threads():
    """Calls of one object from two host threads on one stream: a lock keeps a call's launches together."""
    T, d = 300, 520
    g = gen(3)
    n = LayerNorm(randn(g, d), randn(g, d))
    ns = NewtonSchulz(1, 200, 300)
    n.reserve_backward()
    xs, dys, Gs = ([randn(g, *s) for _ in range(2)] for s in ((T, d), (T, d), (1, 200, 300)))
    stats = [(torch.empty(T, device="cuda"), torch.empty(T, device="cuda")) for _ in range(2)]
    want = []
    for i in range(2):
        n.forward(xs[i], None, *stats[i])
        out = [torch.empty_like(xs[i]), torch.empty(d, device="cuda"), torch.empty(d, device="cuda")]
        n.backward(dys[i], xs[i], *stats[i], *out)
        want.append(out + [ns.orthogonalize(Gs[i])])
    torch.cuda.synchronize()
    got = [[[torch.empty_like(t) for t in want[i]] for _ in range(20)] for i in range(2)]
    s = torch.cuda.Stream()
    gate = threading.Barrier(2)

    def work(i):
        gate.wait()
        for out in got[i]:
            n.backward(dys[i], xs[i], *stats[i], *out[:3], stream=s)
            ns.orthogonalize(Gs[i], out[3], stream=s)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    for i in range(2):
        for out in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(out, want[i]))


def test_workspace_is_not_made_in_a_capture():
    x = torch.ones(4, 16, device="cuda")
    n = LayerNorm(torch.ones(16, device="cuda"))
    m = torch.ones(4, device="cuda")
    refusal = None
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        try:
            n.backward(x, x, m, m, None, torch.empty(16, device="cuda"))
        except B.WasteError as e:
            refusal = e
        x.add_(1)
    assert refusal is not None and refusal.status == -1
    del gr


def test_copies():
    """Copies and pickles work on their own."""
    c = Calls(*SHAPES[0])
    c.run()
    want = c.kept()
    for again in (copy.copy, copy.deepcopy, lambda o: pickle.loads(pickle.dumps(o))):
        c.norm, c.grouped, c.ns = again(c.norm), again(c.grouped), again(c.ns)
        c.fill(0)
        c.w, c.b, c.gw = c.norm.weight, c.norm.bias, c.grouped.w
        g = gen(100)
        for t in (c.w, c.b, c.x, c.dy, c.gw, c.gx, c.gdy, c.G):
            t.copy_(randn(g, *t.shape))
        c.run()
        assert same(c.kept(), want)


def test_weights_written_just_before():
    """What another kernel of the stream writes right before a call is what the call reads."""
    c = Calls(*SHAPES[1])
    for i in range(6):
        c.fill(i)
        torch.cuda.synchronize()
        c.run()
        want = c.kept()
        c.fill(i + 1)
        torch.cuda.synchronize()
        c.fill(i)  # not waited for
        c.run()
        assert same(c.kept(), want)


# ---------------------------------------------------------------- sizes past 2^31

def test_norm_of_many_values():
    T, d = 300007, 7168  # 2.15e9 values
    x = torch.empty(T, d, dtype=BF, device="cuda")
    x.normal_(generator=gen(1))
    n = LayerNorm(1 + randn(gen(2), d, scale=0.1), randn(gen(3), d))
    y, mean, rstd = torch.empty_like(x), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    n.forward(x, y, mean, rstd)
    rows = torch.tensor([0, 1, 149000, 299592, 299593, 299594, T - 2, T - 1], device="cuda")
    ref = R.norm_forward(x[rows], n.weight, n.bias, 1e-5, BF)
    R.close(y[rows], *ref["y"], "y")
    dx, dw, db = torch.empty_like(x), torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    n.backward(y, x, mean, rstd, dx, dw, db)
    v, e = R.norm_backward(y[rows], x[rows], mean[rows], rstd[rows], n.weight)["dx"]
    R.close(dx[rows], v, e + R.rnd(v.abs() + e, BF), "dx")
    want = torch.zeros(d, dtype=torch.float64, device="cuda")
    size = torch.zeros(d, dtype=torch.float64, device="cuda")
    for part in y.split(20000):
        want += part.double().sum(0)
        size += part.double().abs().sum(0)
    # chains of T / 152 rows, then 152 partial sums
    assert ((db.double() - want).abs() <= (T / 152 + 200) * R.U * size).all()


def test_grouped_past_31_bits():
    """A stack of matrices, and a batch, of more than 2^31 values."""
    g = gen(4)
    E, n, k = 200, 1536, 7168
    w = torch.empty(E, n, k, dtype=BF, device="cuda")
    w.normal_(generator=g)
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[1:] = 3
    off[E - 2:] = torch.tensor([3, 10, 15], dtype=torch.int32)
    x, dy = randn(g, 15, k, t=BF), randn(g, 15, n, t=BF)
    m = GroupedLinear(w)
    y, dx = m.forward(x, off), torch.empty_like(x)
    m.backward(dy, x, off, dx)
    for rows, e in ((slice(0, 3), 0), (slice(3, 10), E - 2), (slice(10, 15), E - 1)):
        one = torch.tensor([0, rows.stop - rows.start], dtype=torch.int32, device="cuda")
        for a, b, v in ((x, w[e:e + 1], y), (dy, w[e:e + 1].transpose(1, 2), dx)):
            ref, err = R.grouped(a[rows], one, b)
            R.close(v[rows], ref, err + R.rnd(ref.abs() + err, BF), "far matrix")
    dw = torch.empty_like(w)
    m.backward(dy, x, off, None, dw)
    ref, err = R.grouped_weights(dy[10:], x[10:], torch.tensor([0, 5]))
    R.close(dw[E - 1:], ref, err + R.rnd(ref.abs() + err, BF), "far gradient")
    assert (dw[1:E - 2] == 0).all()
    del w, m, dw, y, dx
    rows, k, n = 300000, 7200, 16
    x = torch.empty(rows, k, dtype=BF, device="cuda")
    x.normal_(generator=g)
    w = randn(g, 2, n, k, t=BF)
    off = torch.tensor([0, 7, rows], dtype=torch.int32, device="cuda")
    m = GroupedLinear(w)
    y = m.forward(x, off)
    last = torch.tensor([0, 0, 40], dtype=torch.int32, device="cuda")
    ref, err = R.grouped(x[-40:], last, w)
    R.close(y[-40:], ref, err + R.rnd(ref.abs() + err, BF), "far rows")


# ---------------------------------------------------------------- decode stacks

def workload(tokens, layers=3):
    return synth.Workload("normed", 256, 128, 8, 2, tokens, "f32", "offsets", n_layers=layers, lookahead=2)


@pytest.mark.parametrize("tokens", [1, 3])
def test_stack_with_norms(tokens):
    """A decode stack whose layers have a norm of their own, or none: eager, captured and replayed."""
    w = workload(tokens)
    layers = [MoELayer(w, 1, L, "cuda") for L in range(3)]
    g = gen(50)
    norms = [LayerNorm(1 + randn(g, 256, scale=0.2), randn(g, 256, scale=0.1)), None, LayerNorm((1 + randn(g, 256, scale=0.2)).to(BF))]
    try:
        hidden = [randn(g, tokens, 256) for _ in range(3)]
        main, side = torch.cuda.Stream(), torch.cuda.Stream()
        stack = DecodeStack(layers, tokens, norm=norms)
        want = []
        for h0 in hidden:
            h, x = h0.clone(), torch.empty_like(h0)
            idx, gate, logits, _ = layers[0].alloc_outputs(tokens)
            for L in range(3):
                if norms[L] is None:
                    B.waste_moe_rmsnorm(h, x, tokens, 256)
                else:
                    norms[L].forward(h, x)
                    R.close(x, *R.norm_forward(h, norms[L].weight, norms[L].bias, 1e-5, FP)["y"], "x")
                layers[L].route(x, tokens, idx, gate, logits)
                layers[L].forward(x, tokens, idx, gate, h, 1)
            want.append(h)
            torch.cuda.synchronize()
            out = stack.run(h0, 2, main, side)
            torch.cuda.synchronize()
            assert torch.equal(out, h)
        h0 = hidden[0].clone()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=main):
            out = stack.run(h0, 2, main, side)
        for i in (2, 0, 1):
            h0.copy_(hidden[i])
            gr.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want[i])
        del gr
        with pytest.raises(ValueError):
            DecodeStack(layers, tokens, norm=norms[:2])
        with pytest.raises(ValueError):
            DecodeStack(layers, tokens, norm=[LayerNorm(torch.ones(128, device="cuda"))] * 3)
    finally:
        for m in layers:
            m.close()


# ---------------------------------------------------------------- a training step

def test_training_step():
    """One step of a layer whose experts are still dense: norm, routing, products grouped by expert with the gated block
    between them, the same backwards, and the experts' weights moved by their orthogonalised gradients.  Every operator's
    outputs are held against the plain form on what it was given."""
    T, d, f, E, top = 190, 264, 136, 6, 2
    g = gen(60)
    t = BF
    h = randn(g, T, d)
    norm = LayerNorm(1 + randn(g, d, scale=0.1), randn(g, d, scale=0.1))
    wg, wu = (randn(g, E, f, d, scale=d ** -0.5, t=t) for _ in range(2))
    wd = randn(g, E, d, f, scale=f ** -0.5, t=t)
    gate, up, down = GroupedLinear(wg), GroupedLinear(wu), GroupedLinear(wd)
    router = randn(g, E, d, scale=d ** -0.5)

    def near(got, ref, to):
        v, e = ref
        R.close(got, v, e + R.rnd(v.abs() + e, to), "step")

    # forward
    mean, rstd = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    x = norm.forward(h, torch.empty(T, d, dtype=t, device="cuda"), mean, rstd)
    R.close(x, *R.norm_forward(h, norm.weight, norm.bias, 1e-5, t)["y"], "x")
    idx, weight = torch.empty(T, top, dtype=torch.int32, device="cuda"), torch.empty(T, top, device="cuda")
    B.waste_moe_topk_from_logits(x.float() @ router.T, T, E, top, idx, weight)
    order = torch.argsort(idx.flatten(), stable=True)
    token = order // top
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[1:] = torch.bincount(idx.flatten(), minlength=E).cumsum(0)
    xs = x[token].contiguous()
    gs, us = gate.forward(xs, off), up.forward(xs, off)
    near(gs, R.grouped(xs, off, wg), t)
    near(us, R.grouped(xs, off, wu), t)
    s = torch.sigmoid(gs.float())
    a = (gs.float() * s * us.float()).to(t)
    ys = down.forward(a, off)
    near(ys, R.grouped(a, off, wd), t)
    # backward of sum_t <dy_t, sum_j weight_tj ys>
    dy = randn(g, T, d)
    dys = (dy[token] * weight.flatten()[order][:, None]).to(t)
    da, dwd = torch.empty_like(a), torch.empty_like(wd, dtype=FP)
    down.backward(dys, a, off, da, dwd)
    near(da, R.grouped(dys, off, wd.transpose(1, 2)), t)
    near(dwd, R.grouped_weights(dys, a, off), FP)
    du = (da.float() * gs.float() * s).to(t)
    dg = (da.float() * us.float() * s * (1 + gs.float() * (1 - s))).to(t)
    dxs, dxu = torch.empty_like(xs), torch.empty_like(xs)
    dwg, dwu = (torch.empty_like(wg, dtype=FP) for _ in range(2))
    gate.backward(dg, xs, off, dxs, dwg)
    up.backward(du, xs, off, dxu, dwu)
    near(dwg, R.grouped_weights(dg, xs, off), FP)
    near(dxu, R.grouped(du, off, wu.transpose(1, 2)), t)
    dx = torch.zeros(T, d, device="cuda").index_add_(0, token, dxs.float() + dxu.float()).to(t)
    dh, dw, db = torch.empty_like(h), torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    norm.backward(dx, h, mean, rstd, dh, dw, db)
    ref = R.norm_backward(dx, h, mean, rstd, norm.weight)
    for got, k in ((dh, "dx"), (dw, "dw"), (db, "db")):
        near(got, ref[k], FP)
    # the update: every expert's gate matrix
    before = wg.clone()
    NewtonSchulz(E, f, d).orthogonalize(dwg, wg, scale=-0.02, mode=1)
    for e in range(E):
        o = R.orthogonal(dwg[e])
        far = 1.5 * R.dense_distance(R.orthogonal_rounded(dwg[e]), o) + 1e-5
        want = before[e].double() - 0.02 * o
        assert (wg[e].double() - want).norm() <= R.half(t) * want.norm() + 0.02 * far * o.norm()
    # the moved matrices serve the next step
    near(gate.forward(xs, off), R.grouped(xs, off, wg), t)


def test_first_backwards_of_two_threads():
    """The first backwards of an object, from two host threads at once on one stream given by its handle, which is not the
    one that the workspace is made on: both take the same, and it stays."""
    T, d = 300, 520
    g = gen(7)
    w, b, x, dy = randn(g, d), randn(g, d), randn(g, T, d), randn(g, T, d)
    mean, rstd = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    n = LayerNorm(w, b)
    n.forward(x, None, mean, rstd)
    want = [torch.empty_like(x), torch.empty(d, device="cuda"), torch.empty(d, device="cuda")]
    n.backward(dy, x, mean, rstd, *want)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(20):
        n = LayerNorm(w, b)
        got = [[torch.empty_like(t) for t in want] for _ in range(2)]
        beside, gate = [None, None], threading.Barrier(2)
        torch.cuda.synchronize()

        def work(i):
            gate.wait()
            n.backward(dy, x, mean, rstd, *got[i], stream=s.cuda_stream)
            beside[i] = torch.full((2432 * d,), 255, dtype=torch.uint8, device="cuda")  # what a dropped workspace left free

        threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
        [t.start() for t in threads]
        [t.join() for t in threads]
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for out in got for p, q in zip(out, want)) and all((t == 255).all() for t in beside)


def test_newton_schulz_is_not_made_in_a_capture():
    x, refusal = torch.ones(4, device="cuda"), None
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        try:
            NewtonSchulz(1, 200, 300)
        except B.WasteError as e:
            refusal = e
        x.add_(1)
    assert refusal is not None and refusal.status == -1
    del gr


@pytest.mark.parametrize("lookahead", [0, 2])
@pytest.mark.parametrize("tokens", [1, 3])
def test_banked_stack_with_norms(tokens, lookahead):
    """Layers whose records come through an HBM cache that evicts, with norms of their own: the resident stack's bits."""
    w = workload(tokens)
    g = gen(51)
    norms = [LayerNorm(1 + randn(g, 256, scale=0.2), randn(g, 256, scale=0.1)), None, LayerNorm((1 + randn(g, 256, scale=0.2)).to(BF))]
    hidden = [randn(g, tokens, 256) for _ in range(3)]

    def run(layers, **k):
        main, side, outs = torch.cuda.Stream(), torch.cuda.Stream(), []
        stack = DecodeStack(layers, tokens, **k)
        torch.cuda.synchronize()
        for h in hidden:
            out = stack.run(h, lookahead, main, side)
            torch.cuda.synchronize()
            outs.append(out.clone())
        return outs

    layers = [MoELayer(w, 1, L, "cuda") for L in range(3)]
    try:
        want, plain = run(layers, norm=norms), run(layers)
    finally:
        for m in layers:
            m.close()
    ts = TieredStack(w, 1, 3, 7)
    try:
        got = run(ts.layers, banked=True, norm=norms)
        assert all(torch.equal(a, b) and not torch.equal(a, c) for a, b, c in zip(got, want, plain))
        for m in ts.layers:
            m.stats()
    finally:
        ts.close()


def test_streams_at_once():
    """Every operator on three streams at the same time, each with objects of its own: the bits of calls alone."""
    calls = [Calls(*s) for s in (SHAPES[1], SHAPES[2], SHAPES[1])]
    want = []
    for i, c in enumerate(calls):
        c.fill(i)
        c.run()
        want.append(c.kept())
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(10):
        for c in calls:
            for t in c.out.values():
                t.fill_(3.0)
        torch.cuda.synchronize()
        for _ in range(5):
            for c, s in zip(calls, streams):
                c.run(s)
        torch.cuda.synchronize()
        assert all(same(c.kept(), w) for c, w in zip(calls, want))

"""The gated feed-forward block, forward and backward, and microscaled 4-bit matrices, their
product and the block on them, against plain 64-bit forms (dense_ref: bounds derived from the
roundings each operator documents)."""
import math

import pytest
import torch

from rvq_compressed_expert_gb300 import binding as B
from rvq_compressed_expert_gb300 import synth
from rvq_compressed_expert_gb300.dense import DenseExpert
from rvq_compressed_expert_gb300.layer import MoELayer
from rvq_compressed_expert_gb300.mx4 import Mx4Expert, Mx4Matrix, matmul
from rvq_compressed_expert_gb300.stack import DecodeStack
from tests import dense_ref as R

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


def guarded(*shape, dtype, fill=7.0):
    """A tensor with 64 rows of a known value behind it, and a check that they were left alone."""
    n = math.prod(shape)
    buf = torch.full((n + 4096,), fill, dtype=dtype, device="cuda")

    def untouched():
        assert (buf[n:] == fill).all()

    return buf[:n].view(*shape), untouched


# d and f of one core matrix, below and past a tile, of no round number, and of the workloads
SHAPES = [(1, 8, 8), (1, 1032, 1544), (2, 64, 24), (3, 256, 128), (5, 264, 1800), (8, 2056, 136), (9, 520, 136), (24, 2056, 1032), (32, 136, 4104), (33, 136, 264), (127, 1032, 136), (128, 512, 520), (129, 72, 1544),
          (150, 2056, 1032), (200, 1032, 264), (208, 4104, 136), (257, 264, 1032), (511, 648, 392), (1000, 1544, 776), (2049, 2056, 1032)]


@pytest.mark.parametrize("t", [BF, HF])
@pytest.mark.parametrize("T,d,f", SHAPES)
def test_forward(T, d, f, t):
    g = gen(T * 7 + d)
    W = weights(g, d, f, t)
    x = randn(g, T, d, t=t)
    e = DenseExpert(*W, max_tokens=T)
    ref = R.forward(x, *W, t)
    out, ok1 = guarded(T, d, dtype=t)
    sg, ok2 = guarded(T, f, dtype=t)
    su, ok3 = guarded(T, f, dtype=t)
    e.forward(x, out, save_g=sg, save_u=su)
    y, ey = ref["y"]
    R.close(out, y, ey + R.rnd(y.abs() + ey, t), "y")
    for n, got in (("g", sg), ("u", su)):
        v, ev = ref[n]
        R.close(got, v, ev + R.rnd(v.abs() + ev, t), n)
    for ok in (ok1, ok2, ok3):
        ok()
    # without g and u, and in fp32, written and added: the same sums
    plain = e.forward(x)
    assert torch.equal(plain, out)
    o32, ok = guarded(T, d, dtype=FP)
    e.forward(x, o32)
    R.close(o32, y, ey + R.rnd(y.abs() + ey, FP), "y in fp32")
    assert torch.equal(o32.to(t), out)
    base = randn(g, T, d)
    acc = base.clone()
    e.forward(x, acc, mode=1)
    R.close(acc, base.double() + y, ey + R.rnd(base.abs().double() + y.abs() + ey, FP), "base + y")
    b16 = base.to(t)
    a16 = b16.clone()
    e.forward(x, a16, mode=1)
    R.close(a16, b16.double() + y, ey + R.rnd(b16.abs().double() + y.abs() + ey, t) + R.rnd(y.abs(), FP), "16-bit base + y")
    ok()


@pytest.mark.parametrize("t", [BF, HF])
@pytest.mark.parametrize("T,d,f", SHAPES)
def test_backward(T, d, f, t):
    g = gen(T * 5 + d)
    W = weights(g, d, f, t)
    x, dy, sg, su = randn(g, T, d, t=t), randn(g, T, d, t=t), randn(g, T, f, t=t), randn(g, T, f, t=t)
    e = DenseExpert(*W, max_tokens=T)
    ref = R.backward(dy, x, sg, su, *W, t)
    dx, ok = guarded(T, d, dtype=t)
    dw, oks = zip(*(guarded(*w.shape, dtype=t) for w in W))
    e.backward(dy, x, sg, su, dx, *dw)
    names = ("dw_gate", "dw_up", "dw_down")
    for n, got in zip(("dx",) + names, (dx,) + dw):
        v, ev = ref[n]
        R.close(got, v, ev + R.rnd(v.abs() + ev, t), n)
    ok()
    for o in oks:
        o()
    # fp32 gradients, added to what is there, dx alone, the weights' alone
    acc = [randn(g, *w.shape) for w in W]
    base = [a.clone() for a in acc]
    e.backward(dy, x, sg, su, None, *acc, accumulate=True)
    for n, got, b in zip(names, acc, base):
        v, ev = ref[n]
        R.close(got, b.double() + v, ev + R.rnd(b.abs().double() + v.abs() + ev, FP), n + " added")
    dx2 = torch.empty_like(dx)
    e.backward(dy, x, sg, su, dx2)
    assert torch.equal(dx2, dx)


def test_backward_is_the_slope():
    """The gradients against central differences of the block itself, in fp64 along random
    directions: (loss(p + h v) - loss(p - h v)) / 2h with loss = <dy, y>."""
    T, d, f, t = 17, 64, 40, HF
    g = gen(3)
    W = weights(g, d, f, t)
    x, dy = randn(g, T, d, t=t), randn(g, T, d, t=t)
    e = DenseExpert(*W, max_tokens=T)
    sg, su = (torch.empty(T, f, dtype=t, device="cuda") for _ in range(2))
    e.forward(x, save_g=sg, save_u=su)
    dx = torch.empty_like(x)
    dw = [torch.empty_like(w, dtype=FP) for w in W]
    e.backward(dy, x, sg, su, dx, *dw)
    P = [x.double(), *(w.double() for w in W)]

    def loss(p):
        gg, uu = p[0] @ p[1].T, p[0] @ p[2].T
        return ((torch.nn.functional.silu(gg) * uu) @ p[3].T * dy.double()).sum()

    for i, got in enumerate([dx, *dw]):
        v = randn(g, *got.shape).double()
        h = 1e-4
        plus, minus = [p.clone() for p in P], [p.clone() for p in P]
        plus[i] += h * v
        minus[i] -= h * v
        slope = float((loss(plus) - loss(minus)) / (2 * h))
        # g, u, a, dg and du each rounded once to fp16 on the way, and dx itself: each moves the
        # result by at most half a step of the magnitudes summed
        scale = float((got.double().abs() * v.abs()).sum())
        assert abs(slope - float((got.double() * v).sum())) <= 6 * R.half(t) * scale + 1e-6 * abs(slope), i


@pytest.mark.parametrize("t", [BF, HF])
def test_no_tokens(t):
    W = weights(gen(1), 64, 32, t)
    e = DenseExpert(*W, max_tokens=4)
    x = torch.empty(0, 64, dtype=t, device="cuda")
    h = torch.empty(0, 32, dtype=t, device="cuda")
    assert e.forward(x).shape == (0, 64)
    dw = [torch.full_like(w, 3.0) for w in W]
    e.backward(x, x, h, h, x.clone(), *dw, accumulate=True)
    assert all((w == 3).all() for w in dw)
    e.backward(x, x, h, h, x.clone(), *dw)
    assert all((w == 0).all() for w in dw)


def test_fewer_tokens_than_reserved_leave_the_rest():
    """T below max_tokens touches the first T rows alone, and nothing of an earlier, longer call
    shows in a shorter one's results."""
    t, d, f = BF, 136, 72
    g = gen(5)
    W = weights(g, d, f, t)
    e = DenseExpert(*W, max_tokens=300)
    big = randn(g, 300, d, t=t)
    big[37:] = float("nan")
    out = torch.full((300, d), 5.0, dtype=t, device="cuda")
    e.forward(big, torch.empty_like(big))
    e.forward(big[:37], out[:37])
    assert (out[37:] == 5).all()
    fresh = DenseExpert(*W, max_tokens=37).forward(big[:37].clone())
    assert torch.equal(fresh, out[:37])
    # one token's result does not depend on the others of its call (same sums, row by row)
    dy, sg, su = randn(g, 300, d, t=t), randn(g, 300, f, t=t), randn(g, 300, f, t=t)
    for v in (dy, sg, su):
        v[37:] = float("nan")
    x = big[:37].contiguous()
    dw = [torch.empty_like(w) for w in W]
    dw2 = [torch.empty_like(w) for w in W]
    e.backward(dy, big, sg, su, None, *dw)
    e.backward(dy[:37], x, sg[:37], su[:37], None, *dw)
    DenseExpert(*W, max_tokens=37).backward(dy[:37], x, sg[:37], su[:37], None, *dw2)
    assert all(torch.equal(a, b) and torch.isfinite(a).all() for a, b in zip(dw, dw2))


def test_past_32_bits():
    """More than 2^31 elements of x and out, and of a matrix to quantise: sampled rows from both ends
    and around the border against the same rows alone."""
    T, d, f, t = 300_000, 7168, 8, BF
    g = gen(77)
    W = weights(g, d, f, t)
    x = torch.empty(T, d, dtype=t, device="cuda")
    for i in range(0, T, 50_000):
        x[i:i + 50_000] = randn(g, 50_000, d, t=t)
    rows = torch.tensor([0, 1, 127, 128, 299_592, 299_593, 299_594, 299_595, T - 129, T - 2, T - 1], device="cuda")
    out = torch.empty_like(x)
    DenseExpert(*W, max_tokens=T).forward(x, out)
    ref = R.forward(x[rows], *W, t)
    y, ey = ref["y"]
    R.close(out[rows], y, ey + R.rnd(y.abs() + ey, t), "y")
    m = Mx4Matrix.from_dense(x)
    code, scale = R.mx_codes(x[rows])
    codes = (code[:, 0::2] + 16 * code[:, 1::2]).to(torch.uint8)
    assert torch.equal(m.codes[rows], codes)
    m.dequantize(out)
    assert torch.equal(out[rows].double(), R.mx_values(code, scale))
    del out, m, x
    torch.cuda.empty_cache()


def test_infinities_and_nans_stay_in_their_rows():
    t, d, f, T = BF, 264, 136, 150
    g = gen(6)
    W = weights(g, d, f, t)
    x = randn(g, T, d, t=t)
    clean = DenseExpert(*W, max_tokens=T).forward(x)
    x[3, 5] = float("nan")
    x[140, 0] = float("inf")
    out = DenseExpert(*W, max_tokens=T).forward(x)
    rows = torch.ones(T, dtype=torch.bool, device="cuda")
    rows[3] = rows[140] = False
    assert torch.isnan(out[3]).all() and not torch.isfinite(out[140]).any()
    assert torch.equal(out[rows], clean[rows])


def test_large_gates():
    """|g| far past the range of exp in fp32: silu is g or 0, its slope 1 or 0."""
    t, d, f, T = BF, 8, 16, 4
    wg = torch.zeros(f, d, dtype=t, device="cuda")
    wg[:8, 0], wg[8:, 0] = 200.0, -200.0
    wu = torch.ones(f, d, dtype=t, device="cuda")
    wd = torch.ones(d, f, dtype=t, device="cuda")
    x = torch.zeros(T, d, dtype=t, device="cuda")
    x[:, 0] = 1.0
    e = DenseExpert(wg, wu, wd, max_tokens=T)
    sg, su = (torch.empty(T, f, dtype=t, device="cuda") for _ in range(2))
    y = e.forward(x, save_g=sg, save_u=su)
    assert (y == 1600).all()
    dw = [torch.empty_like(w) for w in (wg, wu, wd)]
    dx = torch.empty_like(x)
    dy = torch.ones(T, d, dtype=t, device="cuda")
    e.backward(dy, x, sg, su, dx, *dw)
    assert all(torch.isfinite(v).all() for v in (dx, *dw))
    assert (dw[0][:8, 0] == 8 * T).all() and (dw[0][8:] == 0).all() and (dw[2][:, 8:] == 0).all()


@pytest.mark.parametrize("T", [1, 2, 4, 40])
def test_far_gates_leave_nothing(T):
    """Gates of -1000 beside values of 1e30: silu and its slope are 0 in fp32, and so is everything made
    with them, on the way there too (da u alone is past fp32)."""
    t, d, f = BF, 32, 32
    x = torch.zeros(T, d, dtype=t, device="cuda")
    x[:, 0] = 1.0
    wg, wu = (torch.zeros(f, d, dtype=t, device="cuda") for _ in range(2))
    wg[:, 0], wu[:, 0] = -1000.0, 1e30
    wd = torch.ones(d, f, dtype=t, device="cuda")
    e = DenseExpert(wg, wu, wd, max_tokens=T)
    sg, su = (torch.empty(T, f, dtype=t, device="cuda") for _ in range(2))
    assert (e.forward(x, save_g=sg, save_u=su) == 0).all()
    out = [torch.full_like(v, 7.0) for v in (x, wg, wu, wd)]
    e.backward(torch.full_like(x, 1e9), x, sg, su, *out)
    assert all((v == 0).all() for v in out)
    assert (Mx4Expert.from_dense(wg, wu, wd, max_tokens=T).forward(x) == 0).all()


@pytest.mark.parametrize("T", [2, 8, 32, 40])
def test_past_fp16_is_infinite(T):
    """a, du and dg past fp16's range in one column: infinities in what they enter (all other factors are
    positive), and nowhere else."""
    t, d, f = HF, 64, 64
    x = torch.ones(T, d, dtype=t, device="cuda")
    w = torch.full((f, d), 2.0 ** -6, dtype=t, device="cuda")
    w[0] = 8.0
    wd = torch.full((d, f), 0.5, dtype=t, device="cuda")
    e = DenseExpert(w, w, wd, max_tokens=T)
    sg, su = (torch.empty(T, f, dtype=t, device="cuda") for _ in range(2))
    y = e.forward(x, torch.empty(T, d, device="cuda"), save_g=sg, save_u=su)
    assert torch.isposinf(y).all()
    assert (sg[:, 0] == 512).all() and (su[:, 1:] == 1).all()
    dx, dwg, dwu, dwd = (torch.empty_like(v) for v in (x, w, w, wd))
    e.backward(torch.full_like(x, 8.0), x, sg, su, dx, dwg, dwu, dwd)
    assert torch.isposinf(dx).all()
    for v in (dwg, dwu, dwd.T):
        assert torch.isposinf(v[0]).all() and torch.isfinite(v[1:]).all()


def test_expert_refusals():
    g = gen(2)
    W = weights(g, 64, 32, BF)
    e = DenseExpert(*W, max_tokens=4)
    x = randn(g, 4, 64, t=BF)
    bad = [lambda: e.forward(randn(g, 5, 64, t=BF)), lambda: e.forward(x.to(HF)), lambda: e.forward(x.cpu()),
           lambda: e.forward(randn(g, 64, 4, t=BF).T), lambda: e.forward(randn(g, 4, 72, t=BF)),
           lambda: e.forward(x, torch.empty(4, 64, dtype=HF, device="cuda")), lambda: e.forward(x, mode=1),
           lambda: e.forward(x, torch.empty_like(x), mode=3),
           lambda: e.forward(x, save_g=torch.empty(4, 32, dtype=BF, device="cuda")),
           lambda: e.forward(randn(g, 4 * 64 + 1, t=BF)[1:].view(4, 64)),  # 2 bytes past an aligned address
           lambda: e.backward(x, x, x, x, x), lambda: DenseExpert(W[0], W[1], W[0], 4),
           lambda: DenseExpert(*(w.float() for w in W), 4), lambda: DenseExpert(*(w.cpu() for w in W), 4),
           lambda: DenseExpert(*W, 0), lambda: DenseExpert(*weights(g, 60, 32, BF), 4)]
    for call in bad:
        with pytest.raises(B.WasteError) as ei:
            call()
        assert ei.value.status == -1
    h = torch.empty(4, 32, dtype=BF, device="cuda")
    with pytest.raises(B.WasteError):
        e.backward(x, x, h, h, None, torch.empty_like(W[0]), None, None)
    with pytest.raises(B.WasteError):
        e.backward(x, x, h, h, None, *(torch.empty_like(w, dtype=HF) for w in W))
    e.forward(x)  # a valid call still works
    torch.cuda.synchronize()


# ---------------------------------------------------------------- 4-bit matrices

def special(rows, cols, t, g):
    """Values over many binades with zeros, borders, saturation, infinities and NaN among them."""
    v = randn(g, rows, cols) * torch.exp2(torch.randint(-12, 9, (rows, cols // 32), generator=g, device="cuda")
                                          .float().repeat_interleave(32, 1))
    v = v.to(t)
    b = v.view(rows, -1, 32)
    n = b.shape[1]
    b[0, 0] = torch.tensor([7, .25, .5, .75, 1.25, 1.75, 2.5, 3.5, 5, 6, -7, -.25, -.75, -1.25, -1.75, -2.5, -3.5, -5,
                            -0.0, 0, 4, -4, .2499, .2501, 4.999, 5.001, 1, 2, 3, -1, -2, -3], device="cuda").to(t)
    b[-1, -1] = 0
    if rows > 2:
        b[1, n // 2, 3] = float("inf")
        b[2, 0, 31] = float("nan")
        b[1, 0] = torch.finfo(t).max
        b[2, n - 1] = torch.finfo(t).smallest_normal * torch.finfo(t).eps  # smallest subnormal
        b[2, n - 1, 7] = torch.finfo(t).smallest_normal
        b[1, n - 1] = -0.0
    return v


@pytest.mark.parametrize("t", [FP, BF, HF])
@pytest.mark.parametrize("rows,cols", [(1, 32), (1, 7168), (3, 96), (31, 128), (128, 160), (129, 416), (300, 1056)])
def test_quantize_exact(rows, cols, t):
    g = gen(rows + cols)
    x = special(rows, cols, t, g)
    m = Mx4Matrix.empty(rows, cols)
    m.codes.fill_(0xAB)
    m.scales.fill_(0xCD)
    m.quantize(x)
    code, scale = R.mx_codes(x)
    codes, scales = R.mx_pack(code, scale)
    assert torch.equal(m.scales, scales)
    assert torch.equal(m.codes, codes)
    values = R.mx_values(code, scale)
    for o in (FP, BF, HF):
        got = m.dequantize(dtype=o)
        assert torch.equal(torch.isnan(got), torch.isnan(values))
        assert torch.equal(got.nan_to_num(nan=9.0, posinf=1e30, neginf=-1e30),
                           values.to(o).nan_to_num(nan=9.0, posinf=1e30, neginf=-1e30))


def test_quantize_every_exponent():
    """Blocks at every exponent of fp32, subnormals and the largest among them."""
    e = torch.arange(-149, 128, device="cuda", dtype=torch.float64)
    base = torch.tensor([1, -1.5, 1.75, 1.25, -1.875, 0.5, 0.375, 0.125], device="cuda", dtype=torch.float64).repeat(4)
    x = (torch.exp2(e)[:, None] * base).float()
    m = Mx4Matrix.from_dense(x)
    code, scale = R.mx_codes(x)
    codes, scales = R.mx_pack(code, scale)
    assert torch.equal(m.codes, codes) and torch.equal(m.scales, scales)
    assert torch.equal(m.dequantize().double(), R.mx_values(code, scale))


def test_quantize_strided_rows():
    """Rows further apart than their length, in and out; what lies between them stays."""
    g = gen(9)
    wide = randn(g, 70, 256, t=BF)
    x = wide[:, 64:160]
    m = Mx4Matrix.empty(70, 96)
    m.quantize(x)
    codes, scales = R.mx_pack(*R.mx_codes(x))
    assert torch.equal(m.codes, codes) and torch.equal(m.scales, scales)
    back = torch.full((70, 256), 5.0, device="cuda")
    m.dequantize(back[:, 128:224])
    assert torch.equal(back[:, 128:224].double(), R.mx_round(x))
    assert (back[:, :128] == 5).all() and (back[:, 224:] == 5).all()
    one = randn(g, 1, 99, t=HF)[:, :96]  # a single row's stride does not matter
    m1 = Mx4Matrix.from_dense(one)
    assert torch.equal(m1.dequantize().double(), R.mx_round(one))


MATMULS = [(1, 1, 32), (1, 130, 7168), (1, 5001, 1056), (1, 7, 24064), (1, 19000, 7168), (2, 17, 96), (2, 130, 12064), (2, 5001, 1056), (2, 999, 416), (3, 130, 7168), (16, 64, 160), (100, 129, 128), (128, 256, 256), (129, 257, 288),
           (300, 200, 1056), (257, 1000, 512), (640, 513, 2048), (1000, 1100, 544), (2500, 2100, 1056)]


@pytest.mark.parametrize("M,N,K", MATMULS)
def test_matmul(M, N, K):
    g = gen(M + N + K)
    A, Bm = randn(g, M, K), randn(g, N, K)
    A *= torch.exp2(torch.randint(-6, 7, (M, K // 32), generator=g, device="cuda").float()).repeat_interleave(32, 1)
    a, b = Mx4Matrix.from_dense(A), Mx4Matrix.from_dense(Bm)
    va, vb = R.mx_round(A), R.mx_round(Bm)
    ref = va @ vb.T
    err = (va.abs() @ vb.abs().T) * (K * R.SUM)
    for t in (FP, BF, HF):
        out, ok = guarded(M, N, dtype=t)
        matmul(a, b, out)
        R.close(out, ref, err + R.rnd(ref.abs() + err, t), t)
        ok()
        base = randn(g, M, N, t=t)
        acc = base.clone()
        matmul(a, b, acc, mode=1)
        R.close(acc, base.double() + ref, err + R.rnd(base.abs().double() + ref.abs() + err, t) + R.rnd(ref.abs(), FP),
                f"{t} added")
    assert torch.equal(matmul(a, b), matmul(a, b))


def test_matmul_extreme_scales():
    """Scales whose products come near fp32's largest and smallest normal numbers, and a matrix times
    itself."""
    x = torch.ones(40, 64, device="cuda")
    x[:20] *= 2.0 ** 60
    x[20:] *= 2.0 ** -60
    a = Mx4Matrix.from_dense(x)
    ref = x.double() @ x.double().T
    out = matmul(a, a)
    assert torch.equal(out.double(), ref)


def test_matmul_nan_blocks():
    """A NaN block makes NaN of its row (A) or column (B) alone."""
    g = gen(12)
    A, Bm = randn(g, 140, 96), randn(g, 150, 96)
    clean = matmul(Mx4Matrix.from_dense(A), Mx4Matrix.from_dense(Bm))
    A[130, 40], Bm[7, 95] = float("nan"), float("inf")
    out = matmul(Mx4Matrix.from_dense(A), Mx4Matrix.from_dense(Bm))
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[130], bad[:, 7] = True, True
    assert torch.isnan(out[bad]).all() and torch.equal(out[~bad], clean[~bad])


def mx4_block(x, W, t_out):
    """(y, bound) of the 4-bit block for x, from fp64 sums."""
    f, d = W[0].shape
    vx, vg, vu, vd = R.mx_round(x), *(R.mx_round(w) for w in W)
    g, u = vx @ vg.T, vx @ vu.T
    eg, eu = ((vx.abs() @ v.abs().T) * (d * R.SUM) for v in (vg, vu))
    s = torch.sigmoid(g)
    a = g * s * u
    ea = 1.1 * eg * (u.abs() + eu) + (g * s).abs() * eu + R.FUN * a.abs()
    q, dq = R.mx_round(a), R.mx_spread(a, ea)
    y = q @ vd.T
    return y, dq @ vd.abs().T + ((q.abs() + dq) @ vd.abs().T) * (f * R.SUM)


@pytest.mark.parametrize("tx,to", [(FP, FP), (BF, BF), (HF, FP)])
@pytest.mark.parametrize("T,d,f", [(1, 32, 32), (1, 4128, 160), (1, 26624, 64), (2, 64, 26624), (2, 160, 2080), (3, 288, 96), (4, 1056, 160), (5, 256, 128), (8, 6176, 1056), (130, 288, 416), (260, 512, 352), (1000, 1184, 800)])
def test_mx4_expert(T, d, f, tx, to):
    g = gen(T + d + f)
    W = weights(g, d, f, BF)
    x = randn(g, T, d, t=tx)
    e = Mx4Expert.from_dense(*W, max_tokens=T)
    y, ey = mx4_block(x, W, to)
    out, ok = guarded(T, d, dtype=to)
    e.forward(x, out)
    R.close(out, y, ey + R.rnd(y.abs() + ey, to), "y")
    ok()
    base = randn(g, T, d)
    acc = base.clone()
    e.forward(x, acc, mode=1)
    R.close(acc, base.double() + y, ey + R.rnd(base.abs().double() + y.abs() + ey, FP), "base + y")


def test_mx4_refusals():
    g = gen(4)
    W = weights(g, 64, 32, BF)
    m = [Mx4Matrix.from_dense(w) for w in W]
    e = Mx4Expert(*m, max_tokens=2)
    x = randn(g, 2, 64)
    bad = [lambda: Mx4Matrix.empty(4, 48), lambda: Mx4Matrix.from_dense(x.double()), lambda: Mx4Matrix.from_dense(x.cpu()),
           lambda: Mx4Matrix.from_dense(randn(g, 64, 2).T), lambda: Mx4Matrix.from_dense(randn(g, 4, 66)[:, 2:]),
           lambda: Mx4Matrix(32, 64, m[0].codes, m[0].scales[:-1]), lambda: Mx4Matrix(32, 96, m[0].codes, m[0].scales),
           lambda: m[0].quantize(x), lambda: m[0].dequantize(x), lambda: matmul(m[0], m[2]),
           lambda: matmul(m[0], m[1], mode=1), lambda: matmul(m[0], m[1], torch.empty(32, 31, device="cuda")),
           lambda: matmul(m[0], m[1], torch.empty(32, 32, device="cuda"), mode=4),
           lambda: Mx4Expert(m[0], m[2], m[1], 2), lambda: Mx4Expert(*m, max_tokens=0), lambda: e.forward(randn(g, 3, 64)),
           lambda: e.forward(x, torch.empty(2, 96, device="cuda")), lambda: e.forward(x, mode=1), lambda: e.forward(x.cpu())]
    for call in bad:
        with pytest.raises(B.WasteError) as ei:
            call()
        assert ei.value.status == -1
    e.forward(x)
    B.waste_dense_status()  # waits; no device wait gave up


# ---------------------------------------------------------------- as they are used together

def run_captured(fn):
    """fn's work recorded into a graph (after one eager call) and replayed twice."""
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fn()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        fn()
    return gr


def test_training_step_then_four_bits():
    """A dense expert is trained for a step in a captured graph (forward, backward, update of its
    own weights), then quantised and served in 4 bits: each stage against its 64-bit form on
    the very same inputs."""
    t, T, d, f = BF, 96, 320, 224
    g = gen(21)
    W = list(weights(g, d, f, t))
    x, target = randn(g, T, d, t=t), randn(g, T, d, t=t)
    e = DenseExpert(*W, max_tokens=T)
    e.reserve_backward()
    y, sg, su = torch.empty_like(x), *(torch.empty(T, f, dtype=t, device="cuda") for _ in range(2))
    dx, dy = torch.empty_like(x), torch.empty_like(x)
    dw = [torch.zeros(w.shape, device="cuda") for w in W]

    def step():
        e.forward(x, y, save_g=sg, save_u=su)
        torch.sub(y, target, out=dy)
        e.backward(dy, x, sg, su, dx, *dw)

    gr = run_captured(step)
    for v in (y, sg, su, dx, dy, *dw):
        v.fill_(float("nan"))
    gr.replay()
    ref = R.backward(dy, x, sg, su, *W, t)
    for n, got, o in (("dx", dx, t), ("dw_gate", dw[0], FP), ("dw_up", dw[1], FP), ("dw_down", dw[2], FP)):
        v, ev = ref[n]
        R.close(got, v, ev + R.rnd(v.abs() + ev, o), n)
    for w, v in zip(W, dw):
        w.sub_(0.1 * v)  # the expert borrows its weights: the next call uses the new ones
    gr.replay()
    yr, ey = R.forward(x, *W, t)["y"]
    R.close(y, yr, ey + R.rnd(yr.abs() + ey, t), "y after the update")
    q = Mx4Expert.from_dense(*W, max_tokens=T)
    out = q.forward(x)
    y4, e4 = mx4_block(x, W, t)
    R.close(out, y4, e4 + R.rnd(y4.abs() + e4, t), "4-bit y")


def test_streams_and_graphs():
    """Calls on a side stream, two experts on two streams at once, and captured calls replayed on
    new inputs give the bits of plain calls."""
    g = gen(30)
    t, T, d, f = BF, 70, 640, 416
    W = weights(g, d, f, t)
    xs = [randn(g, T, d, t=t) for _ in range(2)]
    dense = [DenseExpert(*W, max_tokens=T) for _ in range(2)]
    four = [Mx4Expert.from_dense(*W, max_tokens=T) for _ in range(2)]
    want = [(dense[0].forward(x).clone(), four[0].forward(x).clone()) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [[torch.empty_like(xs[0]) for _ in range(2)] for _ in range(2)]
    for _ in range(20):
        for i, s in enumerate(streams):
            dense[i].forward(xs[i], outs[i][0], stream=s)
            four[i].forward(xs[i], outs[i][1], stream=s)
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(outs[i][0], want[i][0]) and torch.equal(outs[i][1], want[i][1])
    x = xs[0].clone()
    o = [torch.empty_like(x) for _ in range(2)]

    def both():
        dense[0].forward(x, o[0])
        four[0].forward(x, o[1])

    gr = run_captured(both)
    for i in (1, 0, 1):
        x.copy_(xs[i])
        gr.replay()
        torch.cuda.synchronize()
        assert torch.equal(o[0], want[i][0]) and torch.equal(o[1], want[i][1])


@pytest.mark.parametrize("T,d,f", [(3, 2048, 768), (20, 1920, 608), (131, 4096, 1024), (300, 1024, 288)])
def test_repeats_give_the_same_bits(T, d, f):
    """Calls one behind another, with another stream's work beside some of them: every output's bits are the
    first call's (split sums meet in one order, whoever is first)."""
    g = gen(T + d)
    t = BF
    W = weights(g, d, f, t)
    e, q = DenseExpert(*W, max_tokens=T), Mx4Expert.from_dense(*W, max_tokens=T)
    x, dy = randn(g, T, d, t=t), randn(g, T, d, t=t)
    side, other = torch.cuda.Stream(), torch.zeros(1 << 26, device="cuda")
    want, differ = None, torch.zeros((), dtype=torch.int64, device="cuda")
    for i in range(60):
        if i % 3 == 0:
            with torch.cuda.stream(side):
                other.add_(1)
        got = [torch.full_like(v, float("nan")) for v in (x, x, x, *W)]
        sg, su = (torch.full((T, f), float("nan"), dtype=t, device="cuda") for _ in range(2))
        e.forward(x, got[0], save_g=sg, save_u=su)
        q.forward(x, got[1])
        e.backward(dy, x, sg, su, *got[2:])
        want = want or got
        differ += ~torch.stack([(a == b).all() for a, b in zip(got, want)]).all()
    assert int(differ) == 0
    side.synchronize()


@pytest.mark.parametrize("T", [1, 7, 40, 300])
def test_backward_captured(T):
    """A captured backward, replayed on other inputs, gives the bits of a plain one; called through a
    current stream that is not the one the expert was made on."""
    t, d, f = HF, 392, 264
    g = gen(50 + T)
    W = weights(g, d, f, t)
    e = DenseExpert(*W, max_tokens=T)
    e.reserve_backward()
    sets = [[randn(g, T, n, t=t) for n in (d, d, f, f)] for _ in range(2)]
    want = []
    for s in sets:
        dx, dw = torch.empty(T, d, dtype=t, device="cuda"), [torch.empty_like(w) for w in W]
        e.backward(*s, dx, *dw)
        want.append([dx, *dw])
    buf = [v.clone() for v in sets[0]]
    got = [torch.empty_like(v) for v in want[0]]
    gr = run_captured(lambda: e.backward(*buf, *got))
    for i in (1, 0):
        for a, b in zip(buf, sets[i]):
            a.copy_(b)
        gr.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want[i]))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for v in got:
            v.zero_()
        e.backward(*sets[1], *got)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want[1]))
    fresh = DenseExpert(*W, max_tokens=T)
    gr2 = torch.cuda.CUDAGraph()
    refusal = None
    with torch.cuda.graph(gr2):
        try:
            fresh.backward(*buf, *got)  # would make its workspace inside the capture
        except B.WasteError as err:
            refusal = err
        got[0].zero_()
    assert refusal is not None and refusal.status == -1


@pytest.mark.parametrize("tokens", [1, 3])
def test_stack_with_shared_experts(tokens):
    """A decode stack whose layers have a dense expert, a 4-bit one, and none: every layer's residual
    moves by the routed experts (as without shared ones) plus the shared expert's own output."""
    w = synth.Workload("shared", 256, 128, 8, 2, tokens, "f32", "offsets", n_layers=3, lookahead=2)
    layers = [MoELayer(w, 1, L, "cuda") for L in range(3)]
    g = gen(40)
    W = weights(g, 256, 128, BF)
    shared = [DenseExpert(*W, max_tokens=tokens), Mx4Expert.from_dense(*W, max_tokens=8), None]
    try:
        h0 = randn(g, tokens, 256)
        main, side = torch.cuda.Stream(), torch.cuda.Stream()
        main.wait_stream(torch.cuda.current_stream())
        got = DecodeStack(layers, tokens, shared=shared).run(h0, 2, main, side)
        torch.cuda.synchronize()
        h, x = h0.clone(), torch.empty_like(h0)
        idx, gate, logits, _ = layers[0].alloc_outputs(tokens)
        for L in range(3):
            B.waste_moe_rmsnorm(h, x, tokens, 256)
            layers[L].route(x, tokens, idx, gate, logits)
            layers[L].forward(x, tokens, idx, gate, h, 1)
            if L == 0:
                shared[0].forward(x.to(BF), h, mode=1)
            if L == 1:
                shared[1].forward(x, h, mode=1)
        torch.cuda.synchronize()
        assert torch.equal(got, h)
        without = DecodeStack(layers, tokens).run(h0, 2, torch.cuda.current_stream(), side)
        torch.cuda.synchronize()
        assert not torch.equal(without, got)
        with pytest.raises(ValueError):
            DecodeStack(layers, tokens, shared=shared[:2])
        with pytest.raises(ValueError):
            DecodeStack(layers, tokens + 8, shared=shared)
    finally:
        for m in layers:
            m.close()

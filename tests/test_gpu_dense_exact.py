"""The dense operators on inputs whose every sum is exact in fp32: whole numbers (times a power of two)
whose magnitudes add up to less than 2^24 units, in any order.  Outputs are compared bit for bit, so a part
of k, a low part or a block that is left out or read twice shows; each test first shows on the 64-bit side
that such a loss would change what is compared.

The sigmoid is exactly 1 in fp32 for gates of 32 and more (exp(-32) < 2^-46, and 1 + 2^-46 rounds to 1), so
silu(g) = g and the slope of silu is 1 there.  A whole number below 2^16 is the sum of two bf16 values, one
below 2^15 of two fp16 values: its rounding, and a rest of at most half a step (2^7 and 2^3 units)."""
import pytest
import torch

from rvq_compressed_expert_gb300 import binding as B
from rvq_compressed_expert_gb300.dense import DenseExpert
from rvq_compressed_expert_gb300.mx4 import Mx4Expert, Mx4Matrix, matmul
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


def whole(g, low, high, *shape):
    """Whole numbers low..high in fp64."""
    return torch.randint(low, high + 1, shape, generator=g, device="cuda").double()


def sparse(g, rows, cols, n, values):
    """[rows, cols] fp64 with n nonzeros a row (of the given values), the first and last column among the
    places that can be hit; the last 32 columns always hold one."""
    n = min(n, cols)
    at = torch.rand(rows, cols, generator=g, device="cuda").topk(n, 1).indices
    last = max(cols - 32, 0) + torch.randint(0, min(32, cols), (rows,), generator=g, device="cuda")
    at[:, 0] = torch.where((at == last[:, None]).any(1), at[:, 0], last)
    v = torch.tensor(values, device="cuda", dtype=torch.float64)
    w = torch.zeros(rows, cols, device="cuda", dtype=torch.float64)
    return w.scatter_(1, at, v[torch.randint(0, len(values), (rows, n), generator=g, device="cuda")])


def same(got, ref, what):
    ref = ref.to(got.dtype)
    assert got.shape == ref.shape and torch.isfinite(got).all(), what
    differ = got != ref
    assert not differ.any(), (what, int(differ.sum()), differ.nonzero()[:4].tolist(), got[differ][:4].tolist(),
                              ref[differ][:4].tolist())


def exact_sums(p, q, unit=1.0):
    """p q^T in fp64, its magnitudes' sum shown to be below 2^24 units."""
    assert float((p.abs() @ q.abs().T).max()) < 2 ** 24 * unit
    return p @ q.T


# ---------------------------------------------------------------- values kept in two 16-bit parts

# k split between CTAs (a few tiles) and not (more tiles than clusters that run at once, or one piece of k),
# tokens at both ends of each padded count
TWO_PARTS = [(T, d, f) for T in (2, 3, 16, 17, 31, 32) for d, f in ((320, 200), (1032, 712), (10248, 136), (520, 64), (64, 9992))]


@pytest.mark.parametrize("t", [BF, HF])
@pytest.mark.parametrize("T,d,f", TWO_PARTS)
def test_forward_keeps_both_parts(T, d, f, t):
    """g = 40 + a sum of at most 8 ones, u a sum of at most 8 values up to 63: a = g u has up to 15 bits, y is a
    sum of at most 200 of them."""
    g = gen(T * 31 + d + f)
    x = whole(g, -1, 1, T, d)
    x[:, 0] = 1
    wg = sparse(g, f, d, 8, [1, -1])
    wg[:, 0] = 40
    wu = sparse(g, f, d, 8, [63, -61, 37, -23, 59])
    wd = sparse(g, d, f, 200, [1, -1])
    G, U = exact_sums(x, wg), exact_sums(x, wu)
    a = G * U
    assert G.min() >= 32 and a.abs().max() < 2 ** 15
    y = exact_sums(a, wd)
    assert not torch.equal(a.to(t).double() @ wd.T, y)  # one rounding of a alone would show
    e = DenseExpert(*(w.to(t) for w in (wg, wu, wd)), max_tokens=T)
    out = torch.full((T, d), float("nan"), device="cuda")
    sg, su = (torch.full((T, f), float("nan"), dtype=t, device="cuda") for _ in range(2))
    e.forward(x.to(t), out, save_g=sg, save_u=su)
    same(sg, G, "g")
    same(su, U, "u")
    same(out, y, "y")
    base = whole(g, -1000, 1000, T, d)
    acc = base.float()
    e.forward(x.to(t), acc, mode=1)
    same(acc, base + y, "base + y")


@pytest.mark.parametrize("t", [BF, HF])
@pytest.mark.parametrize("T,d,f", TWO_PARTS)
def test_backward_keeps_both_parts(T, d, f, t):
    """da a sum of at most 8 values up to 14, g 32..127, u up to 255: a, dg and du have up to 15 bits; dx
    is scaled by a power of two into fp16's range."""
    g = gen(T * 17 + d + f)
    x, dy = whole(g, -3, 3, T, d), whole(g, -1, 1, T, d)
    sg, su = whole(g, 32, 127, T, f), whole(g, -255, 255, T, f)
    wd = sparse(g, f, d, 8, [14, -13, 11, -7]).T.contiguous()
    wg, wu = (sparse(g, d, f, 100, [1, -1]).T.contiguous() * 2.0 ** -8 for _ in range(2))
    da = exact_sums(dy, wd.T)
    a, dg, du = sg * su, da * su, da * sg
    assert all(v.abs().max() < 2 ** 15 for v in (a, dg, du))
    assert float(((dg.abs() @ wg.abs()) + (du.abs() @ wu.abs())).max()) < 2 ** 24 * 2.0 ** -8
    dx = dg @ wg + du @ wu
    assert dx.abs().max() < 65504
    dw = [exact_sums(dg.T, x.T), exact_sums(du.T, x.T), exact_sums(dy.T, a.T)]
    cut = [v.to(t).double() for v in (dg, du, a)]
    assert not torch.equal((cut[0] @ wg + cut[1] @ wu).to(t), dx.to(t))
    assert not any(torch.equal(c, v) for c, v in zip((cut[0].T @ x, cut[1].T @ x, dy.T @ cut[2]), dw))
    e = DenseExpert(*(w.to(t) for w in (wg, wu, wd)), max_tokens=T)
    got = torch.full((T, d), float("nan"), dtype=t, device="cuda")
    gw = [torch.full(v.shape, float("nan"), device="cuda") for v in dw]
    call = [v.to(t) for v in (dy, x, sg, su)]
    e.backward(*call, got, *gw)
    same(got, dx, "dx")
    for n, v, r in zip(("dw_gate", "dw_up", "dw_down"), gw, dw):
        same(v, r, n)
    e.backward(*call, None, *gw, accumulate=True)
    for n, v, r in zip(("dw_gate", "dw_up", "dw_down"), gw, dw):
        if float(r.abs().max()) < 2 ** 23:
            same(v, 2 * r, n + " added")


# ---------------------------------------------------------------- 4-bit products and blocks

MATMULS = [(1, 130, 7168), (1, 5001, 1056), (1, 7, 24064), (1, 19000, 7168), (2, 17, 96), (2, 130, 12064), (2, 5001, 1056),
           (2, 999, 416), (3, 130, 7168), (16, 64, 160), (100, 129, 128), (129, 257, 288), (300, 200, 1056), (257, 1000, 512),
           (640, 513, 2048), (509, 7168, 1536), (2500, 2100, 1056)]


@pytest.mark.parametrize("M,N,K", MATMULS)
def test_matmul_exact(M, N, K):
    """Whole numbers up to 6 with powers of two up to 8: sums below 2^24 in any order."""
    g = gen(M + N * 3 + K)
    grid = torch.tensor([0, 1, -1, 2, -2, 3, -3, 4, -4, 6, -6], dtype=torch.float64, device="cuda")
    A, Bm = (grid[torch.randint(0, 11, s, generator=g, device="cuda")] for s in ((M, K), (N, K)))
    A = A * torch.exp2(torch.randint(0, 4, (M, K // 32), generator=g, device="cuda").double()).repeat_interleave(32, 1)
    ref = exact_sums(A, Bm)
    for k in range(0, K, max(32, K // 256 * 32)):  # every one of these blocks of 32 shows in each output tile
        lost = (A[:, k:k + 32] @ Bm[:, k:k + 32].T) != 0
        assert lost.any()
    a, b = Mx4Matrix.from_dense(A.float()), Mx4Matrix.from_dense(Bm.float())
    out = torch.full((M, N), float("nan"), device="cuda")
    matmul(a, b, out)
    same(out, ref, "fp32")
    o16 = torch.full((M, N), float("nan"), dtype=BF, device="cuda")
    matmul(a, b, o16)
    same(o16, ref, "bf16")
    base = whole(g, -1000, 1000, M, N)
    acc = base.float()
    matmul(a, b, acc, mode=1)
    same(acc, base + ref, "added")


BLOCKS = [(1, 64, 32), (1, 4128, 160), (1, 26624, 64), (1, 7168, 1536), (2, 64, 26624), (2, 160, 2080), (2, 26624, 96), (3, 288, 96),
          (3, 7168, 1536), (4, 1056, 160), (5, 256, 128), (8, 6176, 1056), (64, 7168, 1536), (130, 288, 416), (260, 512, 352),
          (1000, 1184, 800)]


@pytest.mark.parametrize("tx", [FP, BF, HF])
@pytest.mark.parametrize("T,d,f", BLOCKS)
def test_mx4_expert_exact(T, d, f, tx):
    """Gates far above 32 (a large term in the first block and a sum of ones over all the others), u a sum of ones
    over all of d: a = g u exactly, quantised as the 64-bit form does, and y a sum below 2^24 of a's units."""
    g = gen(T + d * 3 + f)
    x, wu, wd = whole(g, -1, 1, T, d), whole(g, -1, 1, f, d), whole(g, -1, 1, d, f)
    wg = whole(g, -1, 1, f, d)
    big = 2.0 ** (11 if d > 4096 else 9)
    x[:, :32], wg[:, :32] = 0, 0
    x[:, 0], wg[:, 0] = 1, big
    wu[:, 0] = 0
    G, U = exact_sums(x, wg), exact_sums(x, wu)
    a = G * U
    assert G.min() >= 32 and a.abs().max() < 2 ** 24
    q = R.mx_round(a)
    scale = R.mx_codes(a)[1].double() - 127  # a block's values are multiples of half its power of two
    units = torch.exp2(scale[q.reshape(T, -1, 32).abs().amax(-1) > 0].min() - 1)
    y = exact_sums(q, wd, float(units))
    assert (y != 0).any() and not torch.equal(q[:, :-32] @ wd[:, :-32].T, y)
    lost = R.mx_round(G * (x[:, :-32] @ wu[:, :-32].T)) @ wd.T
    assert d == 64 or not torch.equal(lost, y)
    e = Mx4Expert.from_dense(*(w.float() for w in (wg, wu, wd)), max_tokens=T)
    out = torch.full((T, d), float("nan"), device="cuda")
    e.forward(x.to(tx), out)
    same(out, y, "y")
    base = whole(g, -4, 4, T, d) * float(units)
    acc = base.float()
    e.forward(x.to(tx), acc, mode=1)
    same(acc, base + y, "base + y")
    if tx != HF:
        o16 = torch.full((T, d), float("nan"), dtype=BF, device="cuda")
        e.forward(x.to(tx), o16)
        same(o16, y, "bf16 y")


@pytest.mark.parametrize("T", [2, 16, 17, 32])
@pytest.mark.parametrize("t", [BF, HF])
def test_what_two_parts_leave(T, t):
    """The stated bound on a value kept in two parts, seen through a unit matrix: 2^-16 of it in bf16; in fp16 2^-22,
    but 2^-25 in all where the rest is subnormal.  a = 40 u with u the sum of a value and a small multiple of another, over
    20 binades; one fp32 rounding of a, none of y (one product a column)."""
    d, f = 136, 64
    g = gen(T)
    x = torch.zeros(T, d, dtype=t, device="cuda")
    x[:, 0] = 1
    x[:, 8:] = (torch.randn(T, 128, generator=g, device="cuda") * torch.exp2(torch.randint(-20, 1, (T, 64), generator=g, device="cuda")
                                                                            .float()).repeat(1, 2)).to(t)
    wg, wu, wd = (torch.zeros(s, dtype=t, device="cuda") for s in ((f, d), (f, d), (d, f)))
    wg[:, 0] = 40
    i = torch.arange(f, device="cuda")
    wu[i, 8 + i], wu[i, 72 + i], wd[i, i] = 1, 2.0 ** -9, 1
    e = DenseExpert(wg, wu, wd, max_tokens=T)
    y = torch.empty(T, d, device="cuda")
    e.forward(x, y)
    u = x[:, 8:72].double() + x[:, 72:].double() * 2.0 ** -9
    a = (40 * u.float()).double()
    off = (y[:, :f].double() - a).abs()
    small = a.abs() < 2.0 ** -3
    assert small.any() and (~small).any()
    if t == BF:  # and its least subnormal is far below
        assert (off <= 2.0 ** -16 * a.abs()).all()
    else:
        assert (off <= torch.clamp(2.0 ** -22 * a.abs(), min=2.0 ** -25)).all()
        assert (off > 2.0 ** -22 * a.abs()).any()  # the relative part alone would not hold
    assert (y[:, f:] == 0).all()
    # one part alone is off by far more
    assert ((a.to(t).double() - a).abs() > 8 * off.clamp(min=2.0 ** -30)).any()


@pytest.mark.parametrize("M", [1, 2, 3, 40, 200, 700])
@pytest.mark.parametrize("K", [64, 1056])
def test_matmul_of_extreme_scales(M, K):
    """Ones with every kind of power of two, 2^-127 and 2^127 among them, down to subnormal sums and up past fp32."""
    def ones(rows, byte):
        m = Mx4Matrix.from_dense(torch.ones(rows, K, device="cuda"))  # code 6 is 1 at 2^-2
        real = m.scales == 125
        m.codes.fill_(0x22)
        m.scales[real] = byte
        return m

    for sa, sb in ((0, 127), (0, 240), (1, 250), (0, 254), (254, 0), (100, 20), (60, 60), (57, 57), (53, 53), (50, 58), (254, 254),
                   (190, 190), (189, 189)):
        out = torch.full((M, 200), float("nan"), device="cuda")
        matmul(ones(M, sa), ones(200, sb), out)
        want = torch.tensor(float(K), dtype=torch.float64) * 2.0 ** (sa + sb - 254)
        assert (out == want.float().item()).all(), (sa, sb, out[0, 0].item(), want.item())


# ---------------------------------------------------------------- values that one 16-bit part holds

ONE_PART = [(1, 1032, 1544), (1, 7168, 1536), (33, 136, 264), (48, 2056, 520), (49, 2056, 520), (127, 1032, 136), (128, 512, 520),
            (129, 72, 1544), (131, 7168, 1536), (150, 2056, 1032), (200, 1032, 264), (208, 4104, 136), (209, 4104, 136),
            (257, 264, 1032), (333, 1032, 264), (511, 648, 392), (1000, 1544, 776), (2049, 2056, 1032), (4097, 1032, 1544)]


@pytest.mark.parametrize("t", [BF, HF])
@pytest.mark.parametrize("T,d,f", ONE_PART)
def test_forward_of_whole_numbers(T, d, f, t):
    """Every other column of a has g a sum over all of d (128 and up to 64 ones) and u a power of two, the rest the other
    way round: a has at most 8 bits, so its one rounding is exact, and so is y over all of f."""
    g = gen(T * 13 + d + f)
    x = whole(g, -1, 1, T, d)
    x[:, :2] = 1
    odd = torch.arange(f, device="cuda") % 2 == 1
    wg, wu = (sparse(g, f, d, 64, [1, -1]) for _ in range(2))
    wg[odd], wu[~odd] = 0, 0
    wg[:, :2], wu[:, :2] = 0, 0
    wg[:, 0] = torch.where(odd, 32.0, 128.0)
    wu[~odd, 1] = torch.exp2(whole(g, 0, 4, f))[~odd]
    wd = whole(g, -1, 1, d, f)
    G, U = exact_sums(x, wg), exact_sums(x, wu)
    a = G * U
    assert G.min() >= 32 and torch.equal(a.to(t).double(), a)
    y = exact_sums(a, wd)
    e = DenseExpert(*(w.to(t) for w in (wg, wu, wd)), max_tokens=T)
    out, sg, su = (torch.full((T, n), float("nan"), dtype=o, device="cuda") for n, o in ((d, FP), (f, t), (f, t)))
    e.forward(x.to(t), out, save_g=sg, save_u=su)
    same(out, y, "y")
    same(sg, G, "g")
    same(su, U, "u")
    scaled = wd * 2.0 ** -9  # into fp16's range
    o16 = torch.full((T, d), float("nan"), dtype=t, device="cuda")
    e = DenseExpert(*(w.to(t) for w in (wg, wu, scaled)), max_tokens=T)
    e.forward(x.to(t), o16)
    same(o16, y * 2.0 ** -9, "16-bit y")
    base = whole(g, -1000, 1000, T, d) * 2.0 ** -9
    acc = base.float()
    e.forward(x.to(t), acc, mode=1)
    if float(y.abs().max()) < 2 ** 23:
        same(acc, base + y * 2.0 ** -9, "base + y")


@pytest.mark.parametrize("t", [BF, HF])
@pytest.mark.parametrize("T,d,f", ONE_PART)
def test_backward_of_whole_numbers(T, d, f, t):
    """g and u powers of two, da a sum over all of d of at most 64 ones: a, dg and du have at most 7 bits, and dx and the
    weights' gradients are exact sums over all of f and of the tokens."""
    g = gen(T * 11 + d + f)
    x, dy = whole(g, -1, 1, T, d) * 0.25, whole(g, -1, 1, T, d)
    sg, su = torch.exp2(whole(g, 5, 6, T, f)), torch.exp2(whole(g, 0, 2, T, f)) * (2 * whole(g, 0, 1, T, f) - 1)
    wd = sparse(g, f, d, 64, [1, -1]).T.contiguous()
    wg, wu = (whole(g, -1, 1, f, d) * 2.0 ** -9 for _ in range(2))
    da = exact_sums(dy, wd.T)
    a, dg, du = sg * su, da * su, da * sg
    assert all(torch.equal(v.to(t).double(), v) for v in (a, dg, du))
    assert float(((dg.abs() @ wg.abs()) + (du.abs() @ wu.abs())).max()) < 2 ** 24 * 2.0 ** -9
    dx = dg @ wg + du @ wu
    dw = [exact_sums(dg.T, x.T, 0.25), exact_sums(du.T, x.T, 0.25), exact_sums(dy.T, a.T)]
    e = DenseExpert(*(w.to(t) for w in (wg, wu, wd)), max_tokens=T)
    got = torch.full((T, d), float("nan"), dtype=t, device="cuda")
    gw = [torch.full(v.shape, float("nan"), device="cuda") for v in dw]
    call = [v.to(t) for v in (dy, x, sg, su)]
    e.backward(*call, got, *gw)
    same(got, dx, "dx")
    for n, v, r in zip(("dw_gate", "dw_up", "dw_down"), gw, dw):
        same(v, r, n)
    assert all(v.abs().max() < 65504 for v in dw)
    g16 = [torch.full(v.shape, float("nan"), dtype=t, device="cuda") for v in dw]
    e.backward(*call, None, *g16)
    for n, v, r in zip(("dw_gate", "dw_up", "dw_down"), g16, dw):
        same(v, r, n + " in 16 bits")
    e.backward(*call, None, *gw, accumulate=True)
    for n, v, r in zip(("dw_gate", "dw_up", "dw_down"), gw, dw):
        same(v, 2 * r, n + " added")

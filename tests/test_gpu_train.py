"""Layer norm, products grouped by expert and orthogonalised updates, with their gradients, against plain 64-bit forms
(train_ref: bounds derived from the roundings each operator documents)."""
import math

import pytest
import torch

from rvq_compressed_expert_gb300 import binding as B
from rvq_compressed_expert_gb300.grouped import GroupedLinear
from rvq_compressed_expert_gb300.norm import LayerNorm
from rvq_compressed_expert_gb300.ortho import NewtonSchulz
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


def guarded(*shape, dtype, fill=7.0):
    """A tensor with a known value behind it, and a check that it was left alone."""
    n = math.prod(shape)
    buf = torch.full((n + 4096,), fill, dtype=dtype, device="cuda")

    def untouched():
        assert (buf[n:] == fill).all()

    return buf[:n].view(*shape), untouched


def refused(f, *a, **k):
    with pytest.raises(B.WasteError) as ei:
        f(*a, **k)
    assert ei.value.status == -1


# ---------------------------------------------------------------- layer norm

NORMS = [(1, 1), (3, 7), (1, 7168), (5, 32), (130, 33), (77, 256), (16, 264), (33, 1000), (333, 1001), (9, 4096), (8, 8191), (7, 8192),
         (5, 8200), (3, 16384), (2, 16391), (2, 40000), (2049, 96), (700, 7168)]


def norm_inputs(T, d, tx, tw, seed=0):
    g = gen(T * 31 + d + seed)
    x = randn(g, T, d) * torch.exp(randn(g, 1, d)) + randn(g, T, 1)
    return g, x.to(tx), (1 + randn(g, d, scale=0.2)).to(tw), randn(g, d, t=tw)


@pytest.mark.parametrize("T,d", NORMS)
@pytest.mark.parametrize("tx,ty,tw", [(FP, FP, FP), (BF, BF, BF), (HF, HF, FP), (FP, BF, FP), (BF, FP, HF), (HF, BF, HF)])
def test_norm(T, d, tx, ty, tw):
    g, x, w, b = norm_inputs(T, d, tx, tw)
    n = LayerNorm(w, b)
    y, ok1 = guarded(T, d, dtype=ty)
    mean, ok2 = guarded(T, dtype=FP)
    rstd, ok3 = guarded(T, dtype=FP)
    n.forward(x, y, mean, rstd)
    ref = R.norm_forward(x, w, b, 1e-5, ty)
    for k, got in (("y", y), ("mean", mean), ("rstd", rstd)):
        R.close(got, *ref[k], k)
    again = torch.empty_like(y)
    n.forward(x, again)
    assert torch.equal(again, y)
    dy = randn(g, T, d, t=ty)
    dx, ok4 = guarded(T, d, dtype=tx)
    dw, ok5 = guarded(d, dtype=FP)
    db, ok6 = guarded(d, dtype=FP)
    n.backward(dy, x, mean, rstd, dx, dw, db)
    ref = R.norm_backward(dy, x, mean, rstd, w)
    v, e = ref["dx"]
    R.close(dx, v, e + R.rnd(v.abs() + e, tx), "dx")
    for k, got in (("dw", dw), ("db", db)):
        v, e = ref[k]
        R.close(got, v, e + R.rnd(v.abs() + e, FP), k)
    for ok in (ok1, ok2, ok3, ok4, ok5, ok6):
        ok()
    # each alone gives the same bits; added to what is there; in the weight's type
    only = [torch.empty_like(t) for t in (dx, dw, db)]
    for i in range(3):
        n.backward(dy, x, mean, rstd, *(t if i == j else None for j, t in enumerate(only)))
    assert all(torch.equal(p, q) for p, q in zip(only, (dx, dw, db)))
    base = randn(g, d, t=tw), randn(g, d, t=tw)
    acc = [t.clone() for t in base]
    n.backward(dy, x, mean, rstd, None, *acc, accumulate=True)
    for k, got, b0 in zip(("dw", "db"), acc, base):
        v, e = ref[k]
        v = v + b0.double()
        e = e + R.rnd(v.abs() + e, FP)
        R.close(got, v, e + R.rnd(v.abs() + e, tw), k + " added")


def test_norm_without_weight_or_bias():
    _, x, w, b = norm_inputs(20, 72, BF, BF)
    y = torch.empty(20, 72, device="cuda")
    c = B.waste_norm_config(B.ABI_VERSION, 72, B.ACT_BF16, B.ACT_F32, B.ACT_BF16, 1e-5)
    for pw, pb in ((None, None), (w, None), (None, b)):
        B.waste_norm_forward(c, x, 72, 20, pw, pb, y, 72)
        R.close(y, *R.norm_forward(x, pw, pb, 1e-5, FP)["y"], "y")
    assert torch.equal(LayerNorm(w).forward(x, y.clone()), LayerNorm(w, torch.zeros_like(w)).forward(x, y.clone()))


@pytest.mark.parametrize("t,d,ld", [(BF, 64, 72), (BF, 64, 65), (FP, 40, 44), (FP, 41, 44), (HF, 128, 256), (HF, 7, 9)])
def test_norm_strided_rows(t, d, ld):
    """Rows of a wider tensor; what lies between them stays."""
    T = 21
    g, x, w, b = norm_inputs(T, d, t, FP)
    wide = [torch.full((T, ld), 3.0, dtype=t, device="cuda") for _ in range(4)]
    xs, ys, dys, dxs = (v[:, :d] for v in wide)
    xs.copy_(x)
    dys.copy_(randn(g, T, d))
    n = LayerNorm(w, b)
    mean, rstd = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    n.forward(xs, ys, mean, rstd)
    dw, db = torch.empty(d, device="cuda"), torch.empty(d, device="cuda")
    n.backward(dys, xs, mean, rstd, dxs, dw, db)
    R.close(ys, *R.norm_forward(x, w, b, 1e-5, t)["y"], "y")
    v, e = R.norm_backward(dys, x, mean, rstd, w)["dx"]
    R.close(dxs, v, e + R.rnd(v.abs() + e, t), "dx")
    assert all((v[:, d:] == 3.0).all() for v in wide)
    # two halves of one buffer, in place, dx over dy
    both = torch.cat([x, torch.zeros_like(x)], 1)
    n.forward(both[:, :d], both[:, d:])
    assert torch.equal(both[:, d:], ys) and torch.equal(both[:, :d], x)
    over = x.clone()
    n.forward(over, over)
    assert torch.equal(over, ys)
    over = dys.clone()
    dw2, db2 = torch.empty_like(dw), torch.empty_like(db)
    n.backward(over, xs, mean, rstd, over, dw2, db2)
    assert torch.equal(over, dxs) and torch.equal(dw, dw2) and torch.equal(db, db2)


@pytest.mark.parametrize("d", [1, 5, 8, 9, 33, 1001, 4090, 8185, 8186, 8192])
@pytest.mark.parametrize("tx,ty", [(FP, FP), (BF, BF), (HF, FP), (FP, BF), (BF, HF)])
def test_norm_rows_that_begin_anywhere(tx, ty, d):
    """Each operand at an offset and a stride of its own, so that a row's 16-byte pieces differ between them and from
    row to row; many rows and few."""
    for T, at in ((1301, (1, 3, 6, 5)), (40, (2, 1, 7, 4))):
        g, x, w, b = norm_inputs(T, d, tx, FP)
        bufs = []

        def rows(t, i, values=None):
            ld = d + (1, 2, 5, 3)[i]
            buf = torch.full((at[i] + T * ld + 64,), 7.0, dtype=t, device="cuda")
            v = buf[at[i]:at[i] + T * ld].view(T, ld)[:, :d]
            if values is not None:
                v.copy_(values)
            bufs.append((buf, v))
            return v

        n = LayerNorm(w, b)
        xs, y = rows(tx, 0, x), rows(ty, 1)
        mean, rstd = (torch.empty(T, device="cuda") for _ in range(2))
        n.forward(xs, y, mean, rstd)
        for k, v in (("y", y), ("mean", mean), ("rstd", rstd)):
            R.close(v, *R.norm_forward(x, w, b, 1e-5, ty)[k], k)
        dy = randn(g, T, d, t=ty)
        dys, dx = rows(ty, 2, dy), rows(tx, 3)
        dw, db = (torch.empty(d, device="cuda") for _ in range(2))
        n.backward(dys, xs, mean, rstd, dx, dw, db)
        for k, v, t in (("dx", dx, tx), ("dw", dw, FP), ("db", db, FP)):
            r, e = R.norm_backward(dy, x, mean, rstd, w)[k]
            R.close(v, r, e + R.rnd(r.abs() + e, t), k)
        if tx == ty:  # in place
            n.backward(dys, xs, mean, rstd, dys)
            assert torch.equal(dys, dx)
            n.forward(xs, xs)
            R.close(xs, *R.norm_forward(x, w, b, 1e-5, ty)["y"], "y over x")
        for buf, v in bufs:  # nothing beside the rows
            v.fill_(7.0)
            assert (buf == 7.0).all()


def test_norm_far_values():
    """A mean a thousand times the spread, large and small values, constant rows, rows with an infinity or a NaN."""
    g = gen(5)
    T, d = 24, 1024
    x = randn(g, T, d)
    x[0:4] += 1000.0
    x[4:8] *= 1e15
    x[8:12] *= 1e-12
    x[12:16] = 5.0
    w, b = 1 + randn(g, d, scale=0.1), randn(g, d)
    n = LayerNorm(w, b)
    y, mean, rstd = torch.empty_like(x), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    n.forward(x, y, mean, rstd)
    ref = R.norm_forward(x, w, b, 1e-5, FP)
    R.close(y, *ref["y"], "y")
    R.close(rstd, *ref["rstd"], "rstd")
    assert torch.equal(y[12:16], b.expand(4, d))
    bad = x.clone()
    bad[1, 3], bad[5, 7], bad[17, 1000] = float("inf"), float("nan"), -float("inf")
    z = torch.empty_like(x)
    n.forward(bad, z)
    rows = torch.tensor([1, 5, 17], device="cuda")
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[rows] = False
    assert torch.isnan(z[rows]).all() and torch.equal(z[keep], y[keep])


@pytest.mark.parametrize("T,d", [(5, 1024), (700, 1024), (700, 1001), (3, 16384)])
def test_norm_squares_out_of_range(T, d):
    """Squares about the mean past fp32's range: r is 0 and y is b, as the header says; other rows as ever."""
    g = gen(8)
    x = randn(g, T, d)
    w, b = 1 + randn(g, d, scale=0.1), randn(g, d)
    n = LayerNorm(w, b)
    y, z, mean, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    n.forward(x, y)
    far = x.clone()
    far[1] *= 1e25
    n.forward(far, z, mean, rstd)
    keep = torch.arange(T, device="cuda") != 1
    assert torch.equal(z[1], b) and rstd[1] == 0 and mean[1].isfinite() and torch.equal(z[keep], y[keep])


def test_norm_gradients_are_slopes():
    """Against central differences of the definition in fp64, along random directions."""
    T, d = 6, 40
    g, x, w, b = norm_inputs(T, d, FP, FP)
    dy = randn(g, T, d)
    n = LayerNorm(w, b)
    mean, rstd = torch.empty(T, device="cuda"), torch.empty(T, device="cuda")
    n.forward(x, torch.empty_like(x), mean, rstd)
    grads = [torch.empty_like(t) for t in (x, w, b)]
    n.backward(dy, x, mean, rstd, *grads)
    P = [t.double() for t in (x, w, b)]

    def loss(p):
        c = p[0] - p[0].mean(1, keepdim=True)
        return (dy.double() * (c * (c.square().mean(1, keepdim=True) + 1e-5) ** -0.5 * p[1] + p[2])).sum()

    for i, grad in enumerate(grads):
        v = randn(g, *P[i].shape).double()
        h = 1e-5
        up, down = ([p + s * h * v if i == j else p for j, p in enumerate(P)] for s in (1, -1))
        slope = (loss(up) - loss(down)) / (2 * h)
        # the differences: h^2 of a third derivative of the size of the sum and fp64's 1e-16 / h; the gradient: fp32
        scale = (grad.double() * v).abs().sum()
        assert abs((grad.double() * v).sum() - slope) <= 1e-6 * scale + 1e-7


def test_norm_no_rows():
    w = torch.ones(16, device="cuda")
    n = LayerNorm(w, w)
    x = torch.empty(0, 16, device="cuda")
    none = torch.empty(0, device="cuda")
    assert n.forward(x).shape == (0, 16)
    dw, db = torch.full((16,), 2.0, device="cuda"), torch.full((16,), 2.0, device="cuda")
    n.backward(x, x, none, none, x.clone(), dw, db, accumulate=True)
    assert (dw == 2).all() and (db == 2).all()
    n.backward(x, x, none, none, x.clone(), dw, db)
    assert (dw == 0).all() and (db == 0).all()


def test_norm_refuses():
    w = torch.ones(16, device="cuda")
    n = LayerNorm(w, w)
    x = torch.ones(4, 16, device="cuda")
    m = torch.ones(4, device="cuda")
    refused(LayerNorm, w, w[:8])
    refused(LayerNorm, w, w.half())
    refused(LayerNorm, w.double())
    refused(LayerNorm, w, eps=-1.0)
    refused(LayerNorm, torch.ones(32, device="cuda")[::2])
    for bad in (x[:, :8], x.t(), x.double(), x.cpu(), x[0]):
        refused(n.forward, bad)
        refused(n.forward, x, bad)
        refused(n.backward, bad, x, m, m, x.clone())
    refused(n.forward, x, x[1:])
    refused(n.forward, x, None, m, m[:3])
    refused(n.forward, x, None, m)
    refused(n.forward, x, None, m, m)
    refused(n.backward, x, x, m, m.half(), x.clone())
    refused(n.backward, x, x.clone(), m, m.clone(), x.half())
    refused(n.backward, x, x.clone(), m, m.clone(), None, w.half())
    refused(n.backward, x, x.clone(), m, m.clone(), None, torch.ones(16, device="cuda"), w.half())
    refused(n.backward, x, x.clone(), m, m.clone(), None, w)


# ---------------------------------------------------------------- products grouped by expert

# rows of each expert, k, n
GROUPS = [([1], 8, 8), ([0, 3, 0], 64, 24), ([5, 0, 1, 17, 0, 2, 64, 0], 256, 128), ([128], 72, 264), ([129, 127, 1], 264, 72),
          ([300, 0, 20, 511], 1032, 520), ([0, 0, 0], 64, 64), ([1] * 40, 136, 1032), ([63, 64, 65, 66], 520, 264), ([2049], 136, 520),
          ([16, 15, 1, 0, 200], 7168, 200), ([33, 2, 0, 1000], 200, 1544)]


def group_inputs(sizes, k, n, t, before=0, behind=0, seed=0):
    g = gen(sum(sizes) * 13 + k + n + seed)
    at = [before]
    for s in sizes:
        at.append(at[-1] + s)
    rows = at[-1] + behind
    x, dy = randn(g, rows, k, t=t), randn(g, rows, n, t=t)
    w = randn(g, len(sizes), n, k, scale=k ** -0.5, t=t)
    return g, x, dy, w, torch.tensor(at, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("t", [BF, HF])
@pytest.mark.parametrize("sizes,k,n", GROUPS)
@pytest.mark.parametrize("before,behind", [(0, 0), (3, 70)])
def test_grouped(sizes, k, n, t, before, behind):
    g, x, dy, w, off = group_inputs(sizes, k, n, t, before, behind)
    rows, own = x.shape[0], slice(before, before + sum(sizes))
    if behind:  # what belongs to no expert does not matter, whatever it is
        for v in (x, dy):
            v[:before], v[own.stop:] = float("nan"), float("inf")
    m = GroupedLinear(w)

    def check(got, v, e, to, what, base=7.0):
        R.close(got[own], v[own], e[own] + R.rnd(v[own].abs() + e[own], to), what)
        assert (got[:before] == base).all() and (got[own.stop:] == base).all(), what

    zero = torch.zeros_like
    y, e = R.grouped(torch.where(x.isfinite(), x, zero(x)), off, w)
    for to in (t, FP):
        out, ok = guarded(rows, n, dtype=to)
        out.fill_(7.0)
        m.forward(x, off, out)
        check(out, y, e, to, f"y {to}")
        ok()
        acc = torch.full((rows, n), 7.0, dtype=to, device="cuda")
        m.forward(x, off, acc, mode=1)
        check(acc, y + 7, e + R.rnd(y.abs() + e + 7, FP), to, f"7 + y {to}")
    v, e = R.grouped(torch.where(dy.isfinite(), dy, zero(dy)), off, w.transpose(1, 2))
    dx, ok = guarded(rows, k, dtype=t)
    dx.fill_(7.0)
    for to in (t, FP):
        dw, ok2 = guarded(len(sizes), n, k, dtype=to)
        m.backward(dy, x, off, dx if to == t else None, dw)
        wv, we = R.grouped_weights(dy, x, off)
        R.close(dw, wv, we + R.rnd(wv.abs() + we, to), f"dw {to}")
        ok2()
        base = randn(g, *dw.shape, t=to)
        acc = base.clone()
        m.backward(dy, x, off, None, acc, accumulate=True)
        s = base.double() + wv
        R.close(acc, s, we + R.rnd(s.abs() + we, FP) + R.rnd(s.abs() + 2 * we, to), f"dw added {to}")
        empty = torch.tensor([n == 0 for n in sizes], device="cuda")
        assert (dw[empty] == 0).all() and torch.equal(acc[empty], base[empty])
    check(dx, v, e, t, "dx")
    ok()
    only = torch.full_like(dx, 7.0)
    m.backward(dy, None, off, only)
    assert torch.equal(only, dx)


# sizes whose tiles are wide, by pairs of CTAs ([700, ..]) and by single ones ([100, ..]), and narrow
@pytest.mark.parametrize("t", [BF, HF])
@pytest.mark.parametrize("sizes,k,n", [([37, 0, 130, 1, 16, 300, 63], 456, 328), ([257, 1, 640, 0, 319, 95], 328, 456),
                                       ([1029], 520, 136), ([160] * 40, 72, 1000), ([700, 0, 1, 555, 944], 3336, 4008),
                                       ([100] * 30 + [0, 37], 1304, 2008)])
def test_grouped_exact(t, sizes, k, n):
    """Small whole numbers: every sum is exact, so a lost or a foreign k, row or column shows in the bits."""
    g = gen(1)
    rows = sum(sizes)

    def whole(*shape):
        return torch.randint(-2, 3, shape, generator=g, device="cuda").to(t)

    x, dy, w = whole(rows, k), whole(rows, n), whole(len(sizes), n, k)
    off = torch.tensor([0] + sizes, device="cuda").cumsum(0).to(torch.int32)
    m = GroupedLinear(w)
    y, dx, dw = m.forward(x, off, torch.empty(rows, n, device="cuda")), torch.empty_like(x), torch.empty_like(w, dtype=FP)
    m.backward(dy, x, off, dx, dw)
    assert torch.equal(y.double(), R.grouped(x, off, w)[0])
    assert torch.equal(dw.double(), R.grouped_weights(dy, x, off)[0])
    assert torch.equal(dx, R.grouped(dy, off, w.transpose(1, 2))[0].to(t))


def test_grouped_many_experts():
    """The largest number of experts, most without rows."""
    E, k, n = 4096, 16, 24
    g = gen(9)
    sizes = torch.randint(0, 40, (E,), generator=g, device="cuda") - 34
    off = torch.cat([torch.zeros(1, device="cuda"), sizes.clamp(min=0).cumsum(0)]).to(torch.int32)
    rows = int(off[-1])
    x, dy, w = randn(g, rows, k, t=BF), randn(g, rows, n, t=BF), randn(g, E, n, k, t=BF)
    m = GroupedLinear(w)
    y, e = R.grouped(x, off, w)
    R.close(m.forward(x, off), y, e + R.rnd(y.abs() + e, BF), "y")
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    m.backward(dy, x, off, dx, dw)
    v, e = R.grouped_weights(dy, x, off)
    R.close(dw, v, e + R.rnd(v.abs() + e, BF), "dw")


@pytest.mark.parametrize("sizes,k,n", [([5, 70, 9], 64, 40), ([333, 470, 131], 264, 200), ([500, 470, 431], 2600, 1000)])
def test_grouped_not_finite(sizes, k, n):
    """An infinity or a NaN in a row or a matrix stays with its expert, in the sums over rows too."""
    g, x, dy, w, off = group_inputs(sizes, k, n, BF)
    m = GroupedLinear(w)
    y, dx, dw = m.forward(x, off), torch.empty_like(x), torch.empty_like(w)
    m.backward(dy, x, off, dx, dw)
    x2, dy2 = x.clone(), dy.clone()
    i, j = sizes[0] + 2, sizes[0] + 15  # rows of expert 1
    x2[i, 3], dy2[j, 1] = float("nan"), float("inf")
    y2, dx2, dw2 = m.forward(x2, off), torch.empty_like(x), torch.empty_like(w)
    m.backward(dy2, x2, off, dx2, dw2)
    assert y2[i].isnan().all() and not dx2[j].isfinite().any()
    rows = torch.arange(sum(sizes), device="cuda")
    assert torch.equal(y2[rows != i], y[rows != i]) and torch.equal(dx2[rows != j], dx[rows != j])
    assert torch.equal(dw2[0], dw[0]) and torch.equal(dw2[2], dw[2]) and dw2[1, :, 3].isnan().all()


def test_grouped_bad_offsets():
    """Offsets that fall or leave the rows: nothing outside the buffers is touched, and the status says so."""
    sizes, k, n = [5, 70, 9], 64, 40
    _, x, dy, w, _ = group_inputs(sizes, k, n, BF)
    m = GroupedLinear(w)
    B.waste_dense_status()
    for at in ([0, 5, 75, 85], [0, 5, 3, 84], [-1, 5, 75, 84], [2 ** 31 - 1, -2 ** 31, 0, 84]):
        off = torch.tensor(at, dtype=torch.int32, device="cuda")
        out, ok1 = guarded(84, n, dtype=BF)
        dx, ok2 = guarded(84, k, dtype=BF)
        dw, ok3 = guarded(3, n, k, dtype=BF)
        m.forward(x, off, out)
        with pytest.raises(B.WasteError) as ei:
            B.waste_dense_status()
        assert ei.value.status == -1 and "offsets" in ei.value.message
        B.waste_dense_status()  # said once
        m.backward(dy, x, off, dx, dw)
        with pytest.raises(B.WasteError):
            B.waste_dense_status()
        for ok in (ok1, ok2, ok3):
            ok()


def test_grouped_no_rows():
    w = torch.ones(3, 16, 8, dtype=BF, device="cuda")
    m = GroupedLinear(w)
    x, dy = torch.empty(0, 8, dtype=BF, device="cuda"), torch.empty(0, 16, dtype=BF, device="cuda")
    off = torch.zeros(4, dtype=torch.int32, device="cuda")
    assert m.forward(x, off).shape == (0, 16)
    dw = torch.full((3, 16, 8), 2.0, device="cuda")
    m.backward(dy, x, off, x.clone(), dw, accumulate=True)
    assert (dw == 2).all()
    m.backward(dy, x, off, None, dw)
    assert (dw == 0).all()


def test_grouped_refuses():
    w = torch.ones(3, 16, 8, dtype=BF, device="cuda")
    m = GroupedLinear(w)
    x, dy = torch.ones(6, 8, dtype=BF, device="cuda"), torch.ones(6, 16, dtype=BF, device="cuda")
    off = torch.tensor([0, 1, 2, 6], dtype=torch.int32, device="cuda")
    refused(GroupedLinear, w.float())
    refused(GroupedLinear, w[0])
    refused(GroupedLinear, w.transpose(1, 2))
    for bad in (x.half(), x[:, :4], x.t().contiguous().t(), x[0], x.cpu(), None):
        refused(m.forward, bad, off)
    for bad in (off.long(), off[:3], off.cpu(), None, off.float()):
        refused(m.forward, x, bad)
        refused(m.backward, dy, x, bad, torch.empty_like(x))
    refused(m.forward, x, off, dy[:5])
    refused(m.forward, x, off, dy.half())
    refused(m.forward, x, off, None, 1)
    refused(m.backward, x, x, off, torch.empty_like(x))
    refused(m.backward, dy, None, off, None, torch.empty_like(w))
    refused(m.backward, dy, x, off, x)
    refused(m.backward, dy, x, off, None, w)
    refused(m.backward, dy, x, off, None, torch.empty_like(w, dtype=HF))
    odd = GroupedLinear(torch.ones(2, 12, 8, dtype=BF, device="cuda"))
    refused(odd.forward, x, off[:3].contiguous())


# ---------------------------------------------------------------- orthogonalised updates

def gradient(g, count, rows, cols, rank=None, t=FP):
    if rank is None:
        return randn(g, count, rows, cols, scale=1e-3, t=t)
    return (randn(g, count, rows, rank) @ randn(g, count, rank, cols) * 1e-2).to(t)


def distance(a, b):
    n = b.norm()
    return float((a.double() - b).norm() / n) if n > 0 else float(a.double().norm())


ORTHOS = [(1, 1, 1), (1, 1, 40), (3, 128, 320), (2, 320, 100), (2, 128, 321), (2, 65, 64), (2, 40, 1), (3, 8, 8), (1, 33, 70), (2, 70, 33), (8, 128, 256), (2, 256, 128), (1, 129, 513), (1, 513, 129),
          (1, 264, 1032), (2, 1000, 328), (1, 520, 520), (1, 301, 2007), (3, 201, 1004), (3, 1001, 200)]


@pytest.mark.parametrize("count,rows,cols", ORTHOS)
@pytest.mark.parametrize("t", [FP, BF, HF])
def test_orthogonalize(count, rows, cols, t):
    g = gen(rows * 3 + cols)
    G = gradient(g, count, rows, cols, t=t)
    if t != HF:
        G[0] *= 1e-6 if t == FP else 1e6
    out, ok = guarded(count, rows, cols, dtype=BF)
    NewtonSchulz(count, rows, cols).orthogonalize(G, out)
    ok()
    for z in range(count):
        e = R.orthogonal(G[z])
        # the last rounding (half(BF) of each value), and one and a half times what the documented roundings leave
        assert distance(out[z], e) <= R.half(BF) + 1.5 * distance(R.orthogonal_rounded(G[z]), e) + 1e-5


@pytest.mark.parametrize("rows,cols,rank", [(128, 256, 1), (256, 136, 3), (500, 264, 17), (264, 1032, 64)])
def test_orthogonalize_low_rank(rows, cols, rank):
    """A gradient of fewer tokens than rows: nothing grows outside its space."""
    G = gradient(gen(rank), 1, rows, cols, rank)
    out = NewtonSchulz(1, rows, cols).orthogonalize(G)
    e = R.orthogonal(G[0])
    assert distance(out[0], e) <= R.half(BF) + 1.5 * distance(R.orthogonal_rounded(G[0]), e) + 1e-5
    u = torch.linalg.svd(G[0].double(), full_matrices=False)
    outside = out[0].double() - u[0][:, :rank] @ (u[0][:, :rank].T @ out[0].double())
    assert outside.norm() / e.norm() <= R.half(BF) + 1.5 * distance(R.orthogonal_rounded(G[0]), e) + 1e-5


@pytest.mark.parametrize("rows,cols", [(40, 300), (300, 40), (130, 130), (257, 600), (600, 257)])
def test_orthogonalize_places(rows, cols):
    """One value in each row (or column), at shuffled places: the result has the same places, each the steps of one
    number, and zeros elsewhere."""
    m = min(rows, cols)
    g = gen(rows)
    at = torch.randperm(max(rows, cols), generator=torch.Generator().manual_seed(rows))[:m]
    G = torch.zeros(m, max(rows, cols), device="cuda")
    G[torch.arange(m), at] = torch.where(randn(g, m) > 0, 1.0, -1.0)
    if rows > cols:
        G = G.T.contiguous()
    out = NewtonSchulz(1, rows, cols).orthogonalize(G)
    e = R.orthogonal(G)
    assert torch.equal(out != 0, G != 0)
    s = float(e.abs().max())
    # one number: five steps, each with fp16 roundings of the value (2^-11), its square, and the product; a step
    # makes a relative error at most 3.5 times larger, near the end smaller
    assert (out.double() - e).abs().max() <= (R.half(BF) + 1.5 * distance(R.orthogonal_rounded(G), e) + 1e-4) * s


def test_orthogonalize_added():
    """A weight and its update, in each type; the sum is rounded once."""
    g = gen(2)
    G = gradient(g, 2, 136, 72)
    ns = NewtonSchulz(2, 136, 72)
    e = torch.stack([R.orthogonal(v) for v in G])
    far = max(distance(R.orthogonal_rounded(v), R.orthogonal(v)) for v in G)
    for t in (FP, BF, HF):
        w = randn(g, 2, 136, 72, t=t)
        got = w.clone()
        ns.orthogonalize(G, got, scale=-0.25, mode=1)
        want = w.double() - 0.25 * e
        off = (got.double() - want).norm()
        assert off <= R.half(t) * want.norm() + 0.25 * (1.5 * far + 1e-5) * e.norm()
    a = ns.orthogonalize(G, scale=2.0)
    assert torch.equal(a, (2.0 * ns.orthogonalize(G).double()).to(BF))


@pytest.mark.parametrize("rows,cols", [(64, 96), (96, 64), (136, 200), (330, 96), (130, 131)])
def test_orthogonalize_zero_and_not_finite(rows, cols):
    G = gradient(gen(4), 4, rows, cols)
    ns = NewtonSchulz(4, rows, cols)
    good = ns.orthogonalize(G)
    G[1] = 0.0
    G[2, 5, 5] = float("nan")
    G[3, 1, 2] = float("inf")
    out = ns.orthogonalize(G)
    assert torch.equal(out[0], good[0]) and (out[1] == 0).all() and out[2].isnan().all() and out[3].isnan().all()


@pytest.mark.parametrize("rows,cols", [(48, 80), (140, 88), (90, 400)])
def test_orthogonalize_scales(rows, cols):
    """A power of two times G gives the same bits, however large or small."""
    G = gradient(gen(6), 1, rows, cols)
    ns = NewtonSchulz(1, rows, cols)
    want = ns.orthogonalize(G * 1024)
    for p in (-100, -70, -40, 0, 40, 90, 120):
        assert torch.equal(ns.orthogonalize(G * 1024 * 2.0 ** p), want), p


@pytest.mark.parametrize("steps,abc", [(1, R.MUON), (2, R.MUON), (3, (1.5, -0.5, 0.0)), (8, (1.875, -1.25, 0.375)), (12, R.MUON)])
def test_orthogonalize_steps(steps, abc):
    G = gradient(gen(steps), 1, 96, 200)
    out = NewtonSchulz(1, 96, 200, steps=steps, coefficients=abc).orthogonalize(G[0])
    e = R.orthogonal(G[0], steps, abc)
    assert out.shape == (96, 200)
    assert distance(out, e) <= R.half(BF) + 1.5 * distance(R.orthogonal_rounded(G[0], steps, abc), e) + 1e-5


def test_orthogonalize_refuses():
    refused(NewtonSchulz, 1, 0, 8)
    refused(NewtonSchulz, 1, 8, 8, steps=0)
    refused(NewtonSchulz, 1, 8, 8, coefficients=(9.0, 0.0, 0.0))
    refused(NewtonSchulz, 1, 8, 8, coefficients=(1.0, 2.0))
    ns = NewtonSchulz(2, 8, 16)
    G = torch.ones(2, 8, 16, device="cuda")
    for bad in (G[0], G.double(), G.cpu(), G.transpose(1, 2), None, G[:, :, ::2]):
        refused(ns.orthogonalize, bad)
    refused(ns.orthogonalize, G, G.clone())
    refused(ns.orthogonalize, G, G, mode=1)
    refused(ns.orthogonalize, G, None, mode=1)
    refused(ns.orthogonalize, G, torch.empty(2, 8, 8, dtype=BF, device="cuda"))
    refused(ns.orthogonalize, G, scale=float("nan"))

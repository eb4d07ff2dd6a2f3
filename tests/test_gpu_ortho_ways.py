"""Orthogonalised updates past the small kernel, over every way in which A is made (train_ref.ORTHO_WAYS, pinned without a
GPU by test_train_abi): as a whole and block by block, added to weights of each type, beside zero and not finite ones."""
import pytest
import torch

from rvq_compressed_expert_gb300 import binding as B
from rvq_compressed_expert_gb300.ortho import NewtonSchulz
from tests import train_ref as R

pytestmark = pytest.mark.gpu
BF, HF, FP = torch.bfloat16, torch.float16, torch.float32
WAYS = list(R.ORTHO_WAYS)


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


def gradients(count, rows, cols, t=FP):
    g = torch.Generator("cuda").manual_seed(rows * 3 + cols + count)
    return (torch.randn(count, rows, cols, generator=g, device="cuda") * 1e-3).to(t), g


def blocks(v):
    """Sums over blocks of 32 x 32, the last ones as they are, and how many values each has."""
    rows, cols = v.shape
    p = torch.zeros((rows + 31) // 32 * 32, (cols + 31) // 32 * 32, dtype=torch.float64, device=v.device)
    n = torch.zeros_like(p)
    p[:rows, :cols], n[:rows, :cols] = v, 1
    return tuple(q.view(p.shape[0] // 32, 32, -1, 32).sum((1, 3)) for q in (p, n))


@pytest.mark.parametrize("count,rows,cols", WAYS)
@pytest.mark.parametrize("t", [FP, BF])
def test_whole_and_by_blocks(count, rows, cols, t):
    """The norm as everywhere: the last rounding and one and a half times what the documented ones leave.  Block by block:
    a value's error is a sum of hundreds of roundings, all of one size for a Gaussian gradient, so a block of b values has
    sqrt(b) times their root mean square, four times that at most (and four of them, for the blocks of a few values at an
    edge); one wrong value in a block of 32 x 32 is 8 times more."""
    G, _ = gradients(count, rows, cols, t)
    out = NewtonSchulz(count, rows, cols).orthogonalize(G)
    for z in range(count):
        e = R.orthogonal(G[z])
        far = R.dense_distance(R.orthogonal_rounded(G[z]), e)
        assert R.dense_distance(out[z], e) <= R.half(BF) + 1.5 * far + 1e-5
        rms = (far + 1e-5) * float(e.norm()) / (rows * cols) ** 0.5
        d2, n = blocks((out[z].double() - e).square())
        e2, _ = blocks(e.square())
        assert (d2.sqrt() <= 4 * (n.sqrt() + 1) * rms + R.half(BF) * (e2.sqrt() + 4 * (n.sqrt() + 1) * rms)).all()


@pytest.mark.parametrize("count,rows,cols", WAYS + [(2, 136, 72), (2, 72, 136), (3, 65, 33)])
def test_added(count, rows, cols):
    """Onto weights that are not zero, of each type: what an update onto fp32 zeros holds, added with one rounding, value by
    value; and that update by norm."""
    G, g = gradients(count, rows, cols)
    ns = NewtonSchulz(count, rows, cols)
    alone = torch.zeros(count, rows, cols, device="cuda")
    ns.orthogonalize(G, alone, scale=-0.25, mode=1)
    for z in range(count):
        e = R.orthogonal(G[z])
        far = R.dense_distance(R.orthogonal_rounded(G[z]), e)
        assert R.dense_distance(alone[z], -0.25 * e) <= 1.5 * far + 1e-5
    for t in (FP, BF, HF):
        w = (torch.randn(count, rows, cols, generator=g, device="cuda") * max(rows, cols) ** -0.5).to(t)
        got = w.clone()
        ns.orthogonalize(G, got, scale=-0.25, mode=1)
        want = w.double() + alone.double()
        # the sum in fp32, and its rounding to t (fp16's subnormals: 2^-25)
        bound = R.U * want.abs() + R.rnd(want.abs() * (1 + R.U), t)
        assert ((got.double() - want).abs() <= bound).all(), t


@pytest.mark.parametrize("count,rows,cols", [w for w in WAYS if w[0] >= 3])
def test_zero_and_not_finite_beside(count, rows, cols):
    G, _ = gradients(count, rows, cols)
    ns = NewtonSchulz(count, rows, cols)
    good = ns.orthogonalize(G)
    G[1] = 0.0
    G[2, rows - 1, 5] = float("nan")
    out = ns.orthogonalize(G)
    assert torch.equal(out[0], good[0]) and (out[1] == 0).all() and out[2].isnan().all() and torch.equal(out[3:], good[3:])
    G[2] = float("inf")
    again = ns.orthogonalize(G)
    assert torch.equal(again[:2], out[:2]) and again[2].isnan().all() and torch.equal(again[3:], good[3:])

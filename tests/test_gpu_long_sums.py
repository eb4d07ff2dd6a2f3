"""Products whose sums are so long that a tile of them takes a tenth of a second and more: no bounded wait gives up on
them, and the sums (small whole numbers in few places, exact in any order) are right."""
import pytest
import torch

from rvq_compressed_expert_gb300 import binding as B
from rvq_compressed_expert_gb300.dense import DenseExpert
from rvq_compressed_expert_gb300.grouped import GroupedLinear
from rvq_compressed_expert_gb300.ortho import NewtonSchulz
from tests import train_ref as R

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


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
    torch.cuda.empty_cache()


def gen(seed):
    return torch.Generator("cuda").manual_seed(seed)


def whole(g, *shape):
    return torch.randint(-2, 3, shape, generator=g, device="cuda").to(BF)


def places(g, n):
    """A few hundred of n places, the last ones among them."""
    return torch.cat([torch.randint(0, n, (500,), generator=g, device="cuda"), torch.arange(n - 70, n, device="cuda")]).unique()


def test_forward_of_a_long_k():
    k, n, rows = 1 << 25, 8, 3
    g = gen(1)
    at = places(g, k)
    x, w = torch.zeros(rows, k, dtype=BF, device="cuda"), torch.zeros(1, n, k, dtype=BF, device="cuda")
    x[:, at], w[:, :, at] = whole(g, rows, len(at)), whole(g, 1, n, len(at))
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    y = GroupedLinear(w).forward(x, off, torch.empty(rows, n, device="cuda"))
    B.waste_dense_status()
    assert torch.equal(y.double(), x[:, at].double() @ w[0][:, at].double().T)


def test_dense_gradients_of_many_tokens():
    """The block's dW of 2^28 tokens (gates of 64, whose sigmoid is 1)."""
    T, c = 1 << 28, 8
    g = gen(2)
    at = places(g, T)
    x, dy, u = (torch.zeros(T, c, dtype=BF, device="cuda") for _ in range(3))
    for v in (x, dy, u):
        v[at] = whole(g, len(at), c)
    gate = torch.full((T, c), 64.0, dtype=BF, device="cuda")
    ws = [torch.eye(c, dtype=BF, device="cuda") for _ in range(3)]
    dw = [torch.empty(c, c, device="cuda") for _ in range(3)]
    DenseExpert(*ws, max_tokens=T).backward(dy, x, gate, u, None, *dw)
    B.waste_dense_status()
    p, q, r = dy[at].double(), x[at].double(), u[at].double()
    assert torch.equal(dw[0].double(), (p * r).T @ q)
    assert torch.equal(dw[1].double(), (64 * p).T @ q)
    assert torch.equal(dw[2].double(), p.T @ (64 * r))


@pytest.mark.parametrize("rows", [(1 << 25) - 37, (1 << 30) - 37])
def test_grouped_gradient_of_many_rows(rows):
    """One expert's dW: a tile of a tenth of a second, and of four, whose last piece ends inside rows of no expert."""
    c, behind = 8, 37
    g = gen(3)
    x, dy = (torch.zeros(rows + behind, c, dtype=BF, device="cuda") for _ in range(2))
    at = places(g, rows)
    for v in (x, dy):
        v[at] = whole(g, len(at), c)
        v[rows:] = 3.0  # nobody's
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    w = whole(g, 1, c, c)
    m, dw = GroupedLinear(w), torch.empty(1, c, c, device="cuda")
    m.backward(dy, x, off, None, dw)
    B.waste_dense_status()
    assert torch.equal(dw[0].double(), dy[at].double().T @ x[at].double())
    y = torch.full((rows + behind, c), 7.0, dtype=BF, device="cuda")
    m.forward(x, off, y)
    assert torch.equal(y[at].double(), x[at].double() @ w[0].double().T) and (y[rows:] == 7).all()


def test_grouped_gradient_behind_whole_pieces():
    """Experts of whole pieces of 64 rows, which need no clearing, before one that does, on the same SMs."""
    c, many = 8, (1 << 18) * 64
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    sizes = [many] + [0] * (sms - 1) + [100] + [64] * (sms - 1) + [99]
    off = torch.tensor([0] + sizes, device="cuda").cumsum(0).to(torch.int32)
    rows = int(off[-1])
    g = gen(4)
    x, dy = (torch.zeros(rows, c, dtype=BF, device="cuda") for _ in range(2))
    at = torch.cat([places(g, many), torch.arange(many, rows, device="cuda")])
    for v in (x, dy):
        v[at] = whole(g, len(at), c)
    dw = torch.empty(len(sizes), c, c, device="cuda")
    GroupedLinear(whole(g, len(sizes), c, c)).backward(dy, x, off, None, dw)
    B.waste_dense_status()
    ends = off.tolist()
    for e in range(len(sizes)):
        in_e = at[(at >= ends[e]) & (at < ends[e + 1])] if sizes[e] == many else torch.arange(ends[e], ends[e + 1], device="cuda")
        assert torch.equal(dw[e].double(), dy[in_e].double().T @ x[in_e].double()), e


@pytest.mark.parametrize("rows,cols", [(8, 1 << 28), (1 << 28, 8), (1, 1 << 24), (1 << 24, 1), (3, 5000), (5003, 1)])
def test_orthogonalize_a_long_side(rows, cols):
    """One value on each of the short side's rows, the first and the last place of the long side among them: the steps of one
    number at the same places, zeros elsewhere."""
    m, n = min(rows, cols), max(rows, cols)
    g = gen(5)
    at = places(g, n)
    at = torch.cat([at[:1] * 0, at[torch.randperm(len(at) - 1, generator=g, device="cuda")[:m]], at[-1:]]).unique()
    at = torch.cat([at[:m - 1], at[-1:]]) if m > 1 else at[-1:]
    G = torch.zeros(1, rows, cols, dtype=BF, device="cuda")
    sign = torch.where(torch.arange(m, device="cuda") % 2 == 0, 1.0, -1.0).to(BF)
    i = torch.arange(m, device="cuda")
    G[(0, i, at) if rows <= cols else (0, at, i)] = sign
    out = NewtonSchulz(1, rows, cols).orthogonalize(G)
    B.waste_dense_status()
    small = torch.diag(sign.double())  # the same without the empty places
    e = R.orthogonal(small)
    got = out[0][(i, at) if rows <= cols else (at, i)].double()
    s = float(e.abs().max())
    # as for the shuffled places of a smaller matrix: the last rounding, one and a half times what the documented ones leave
    bound = (R.half(BF) + 1.5 * R.dense_distance(R.orthogonal_rounded(small), e) + 1e-4) * s
    assert (got - torch.diagonal(e)).abs().max() <= bound
    assert int((out != 0).sum()) == m

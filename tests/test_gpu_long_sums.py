"""Products whose sums are so long that a tile of them takes a tenth of a second and more: no bounded wait gives up on
them, and the sums (small whole numbers in few places, exact in any order) are right."""
import pytest
import torch

from rvq_compressed_expert_gb300 import binding as B
from rvq_compressed_expert_gb300.dense import DenseExpert
from rvq_compressed_expert_gb300.grouped import GroupedLinear

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

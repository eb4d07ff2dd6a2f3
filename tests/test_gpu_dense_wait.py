"""The dense operators' bounded device waits: one that nobody ends gives up within about a second, is
reported once, and leaves the GPU usable.  The barrier is the waiting CTA's own: nothing faults or
hangs."""
import time

import pytest
import torch

from rvq_compressed_expert_gb300 import binding as B
from rvq_compressed_expert_gb300.dense import DenseExpert

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from rvq_compressed_expert_gb300 import _build
    _build.build()
    B.load()


def seconds(*a):
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    B.waste_dense_debug_wait(*a)
    torch.cuda.synchronize()
    return time.perf_counter() - t0


def test_a_wait_that_gives_up_is_reported_once():
    B.waste_dense_status()
    W = [torch.ones(64, 64, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    x = torch.full((40, 64), 2.0 ** -6, dtype=torch.bfloat16, device="cuda")
    e = DenseExpert(*W, max_tokens=40)
    want = e.forward(x).clone()
    assert seconds(64) < 0.1
    with pytest.raises(B.WasteError) as ei:
        B.waste_dense_status()
    assert ei.value.status == -6  # WASTE_ETIMEOUT
    B.waste_dense_status()
    assert torch.equal(e.forward(x), want)
    # a wait that is over at once latches nothing
    assert seconds(0, 1) < 0.1
    B.waste_dense_status()


def test_the_operators_limit_is_about_a_second():
    waited = seconds(0)
    with pytest.raises(B.WasteError):
        B.waste_dense_status()
    B.waste_dense_status()
    assert 0.3 < waited < 3.0, waited

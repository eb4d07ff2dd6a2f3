"""What the training operators' Python objects hold between calls: without a GPU, their buffers stood in for."""
import threading
import time
from types import SimpleNamespace

import pytest
import torch

from rvq_compressed_expert_gb300 import _build
from rvq_compressed_expert_gb300 import binding as B
from rvq_compressed_expert_gb300 import norm, ortho


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    B.load()


class Buffer:
    """Stands in for a workspace; making one takes a while, as an allocation does."""

    def __init__(self, nbytes, device):
        time.sleep(0.05)
        self.nbytes = nbytes


def layer_norm(monkeypatch, d=64):
    monkeypatch.setattr(norm, "check", lambda *a: None)
    monkeypatch.setattr(norm, "Workspace", Buffer)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    return norm.LayerNorm(SimpleNamespace(device=torch.device("cuda", 0), dtype=torch.float32, dim=lambda: 1, shape=(d,)))


def test_first_backwards_of_two_threads_share_a_workspace(monkeypatch):
    """Both get the one that the object keeps: another would be dropped while a call's kernels write it."""
    n = layer_norm(monkeypatch)
    gate, got = threading.Barrier(2), []

    def work():
        gate.wait()
        got.append(n.reserve_backward())

    threads = [threading.Thread(target=work) for _ in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    assert len(got) == 2 and got[0] is got[1] is n.reserve_backward()
    assert got[0].nbytes == B.waste_norm_workspace(n._config(torch.float32, torch.float32), 1 << 30)


def test_newton_schulz_is_not_made_in_a_capture(monkeypatch):
    """Its workspace would belong to the graph."""
    made = []
    monkeypatch.setattr(ortho, "Workspace", lambda *a: made.append(a))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    with pytest.raises(B.WasteError) as ei:
        ortho.NewtonSchulz(1, 200, 300, device="cuda:0")
    assert ei.value.status == -1 and "capture" in ei.value.message and not made
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    ortho.NewtonSchulz(1, 200, 300, device="cuda:0")
    assert len(made) == 1

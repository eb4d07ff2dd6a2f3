"""Bounded device waits of the training operators, each unit by its own wait and its own word: one that nobody ends gives
up, is reported once, and leaves the GPU usable.  The barrier is the waiting CTA's own: nothing faults or hangs."""
import time

import pytest
import torch

from rvq_compressed_expert_gb300 import binding as B

pytestmark = pytest.mark.gpu
UNITS = {"norm": 0, "grouped": 1, "ortho": 2}


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
    B.waste_train_debug_wait(*a)
    torch.cuda.synchronize()
    return time.perf_counter() - t0


def gave_up():
    with pytest.raises(B.WasteError) as ei:
        B.waste_dense_status()
    assert ei.value.status == -6  # WASTE_ETIMEOUT
    B.waste_dense_status()  # said once


@pytest.mark.parametrize("unit", UNITS.values(), ids=UNITS)
def test_a_wait_that_gives_up_is_reported_once(unit):
    B.waste_dense_status()
    assert seconds(unit, 64) < 0.1
    gave_up()
    assert seconds(unit, 0, 1) < 0.1  # over at once: latches nothing
    B.waste_dense_status()


def test_all_at_once():
    B.waste_dense_status()
    for unit in UNITS.values():
        seconds(unit, 64)
    seconds(0, 64)
    gave_up()


def test_the_norms_later_waits_are_skipped():
    """Of three waits one behind another the first takes the limit, and the others nothing."""
    waited = seconds(UNITS["norm"])
    gave_up()
    assert 0.3 < waited < 2.0, waited

import gc
import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA GPU (GB300, sm_103a)")


def pytest_collection_finish(session):
    gc.freeze()  # what is imported by now stays: collections between tests are short


@pytest.fixture(autouse=True)
def _garbage_ends_with_its_test():
    """A test's cycles (a caught error and its frames, say) may hold CUDA graphs, and one destroyed by the collector while a
    later test records another makes that recording fail."""
    yield
    gc.collect()


@pytest.fixture(scope="session")
def oracle_mod():
    import oracle
    oracle.build()
    return oracle

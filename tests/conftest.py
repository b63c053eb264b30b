import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs a CUDA device (B200, sm_100a)")
    config.addinivalue_line("markers", "slow: long-running CPU test")


@pytest.fixture(scope="session")
def golden_dir():
    return os.path.join(ROOT, "tests", "golden")


@pytest.fixture(autouse=True)
def structures_outlive_their_addresses(request, monkeypatch):
    """Keeps what a module's cache_struct() makes until its test ends: ctypes.addressof(cache_struct()) alone holds no
    reference, and the library would read memory that may have been given out again."""
    make = getattr(request.module, "cache_struct", None)
    if make is not None:
        kept = []

        def cache_struct(**kw):
            kept.append(make(**kw))
            return kept[-1]
        monkeypatch.setattr(request.module, "cache_struct", cache_struct)
    yield

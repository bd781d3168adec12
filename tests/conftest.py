import os
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)


def pytest_configure(config):
    config.addinivalue_line("markers", "gpu: needs an MI355X (gfx950) GPU and the built HIP library")
    config.addinivalue_line("markers", "slow: long-running host test")


@pytest.fixture(autouse=True)
def _room_behind_arrays(request):
    """The planted mistakes in the oracle read past their arrays (a transposed index does). What follows an array is
    mapped memory then: arrays come from the heap, whose free end is kept larger than any of these overruns."""
    if request.module.__name__ == "test_oracle_mutants":
        import ctypes

        libc = ctypes.CDLL(None)
        libc.malloc.restype, libc.malloc.argtypes, libc.free.argtypes = ctypes.c_void_p, [ctypes.c_size_t], [ctypes.c_void_p]
        trim, threshold = -1, -3                    # M_TRIM_THRESHOLD, M_MMAP_THRESHOLD
        libc.mallopt(trim, 1 << 30)
        libc.mallopt(threshold, 32 << 20)           # the most that it can be
        held = [libc.malloc(24 << 20) for _ in range(8)]
        for block in held:
            libc.free(block)
    yield

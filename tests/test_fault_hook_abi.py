"""The test hook of the bounded waits refuses what it does not know (no GPU needed)."""
import ctypes

import pytest

i64 = ctypes.c_int64


@pytest.fixture(scope="module")
def hook():
    from parity_binade_chunked_gb300 import build
    fn = ctypes.CDLL(build.build()).seqsum_debug_set_fault
    yield lambda mode, arg, wait: fn(ctypes.c_int(mode), i64(arg), i64(wait))
    fn(ctypes.c_int(0), i64(0), i64(0))


def test_modes(hook):
    assert hook(0, 0, 0) == hook(1, 5, 1000) == hook(2, 3 * 128 + 7, 1 << 40) == 0
    for bad in ((-1, 0, 0), (3, 0, 0), (0, 0, -1), (2, -1, 0), (2, 1 << 34, 0)):
        assert hook(*bad) == -1


def test_cluster_sizes(hook):
    assert hook(3, 1, 0) == hook(3, 16, 0) == hook(0, 0, 0) == 0
    for arg in (-1, 0, 17, 1 << 40):
        assert hook(3, arg, 0) == -1

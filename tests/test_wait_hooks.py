"""What the wait-timeout hooks of the windowed decode and the prefill refuse before any launch.  No GPU."""
import ctypes as C
import math

import pytest

import paged_kv_cache_75_gb300 as pk
from paged_kv_cache_75_gb300 import build as pkg_build

FAKE = 1 << 20  # a 16-byte aligned, never dereferenced address


@pytest.fixture(scope="module")
def lib():
    pkg_build.build()
    return pk.library()


def cache():
    return pk._binding._Cache(FAKE, FAKE, 64, 16, 2, 128, pk.PA_F16, 1.0, 1.0)


def test_decode_window_hook(lib):
    def call(n=2, window=8, sinks=2, dt=pk.PA_F16):
        return lib.pa_decode_window_test_wait_timeout(FAKE, FAKE, dt, C.byref(cache()), FAKE, 4, FAKE, n, 64, 4, 0.1, window,
                                                      sinks, 0, None, 0, None, None)
    assert call(window=0) == 1 and call(sinks=-1) == 1 and call(dt=pk.PA_BF16) == 2
    assert call(n=0) == 0


def test_prefill_hook(lib):
    def call(n=2, window=8, sinks=2, dt=pk.PA_F16, scale=0.1):
        return lib.pa_prefill_test_wait_timeout(FAKE, FAKE, dt, C.byref(cache()), FAKE, 4, FAKE, FAKE, n, 8, 64, 4, scale,
                                                window, sinks, None, None)
    assert call(window=-1) == 1 and call(sinks=-1) == 1 and call(scale=0.0) == 1 and call(scale=math.nan) == 1
    assert call(dt=pk.PA_BF16) == 2
    assert call(n=0) == 0 and call(n=0, window=0) == 0

"""The module that marshals the calls of a decode step: what it refuses before any launch.  No GPU."""
import pytest
import torch

import paged_kv_cache_75_gb300 as pk
from paged_kv_cache_75_gb300 import build as pkg_build


@pytest.fixture(scope="module")
def native():
    pkg_build.build()
    return pk._binding._native()


@pytest.mark.parametrize("name,n", [("qk_norm_rope", 6), ("qk_norm_rope_write", 12), ("decode_window", 15),
                                    ("prefill_varlen_window", 15)])
def test_argument_counts_and_kinds(native, name, n):
    f = getattr(native, name)
    for k in (0, n - 1, n + 1):
        with pytest.raises(TypeError, match="arguments expected"):
            f(*[None] * k)
    with pytest.raises(TypeError, match="must be a tensor"):
        f(*[None] * n)
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        f(*[torch.zeros(1, 1, 64, dtype=torch.float16)] * n)
    with pytest.raises(ValueError, match="too many dimensions"):
        f(*[torch.zeros(1, 1, 1, 1, 64, dtype=torch.float16)] * n)


def test_setup_takes_every_function(native):
    with pytest.raises(TypeError):
        native.setup(1, 2)
    with pytest.raises(ValueError):
        native.setup(*[None] * 9, 0, 1, 1, 1)
    pk._binding._native_mod = None  # set up again with the library's own addresses
    assert pk._binding._native() is native


def test_transforms_are_checked_when_made():
    with pytest.raises(ValueError):
        pk.QKTransform(q_weight=torch.ones(2, 64))
    with pytest.raises((TypeError, ValueError)):
        pk.QKTransform(q_weight=torch.ones(64))  # not on a GPU
    t = pk.QKTransform(eps=1e-5, interleaved=True)
    with pytest.raises(Exception):
        t.eps = 1.0

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


class Rows:
    """What the module asks of a tensor."""

    def __init__(self, device):
        self.shape, self.dtype, self.device = (0, 2, 64), torch.float16, device

    def get_device(self):
        return self.device

    def is_contiguous(self):
        return True

    def stride(self):
        return (128, 64, 1)

    def data_ptr(self):
        return 0


def with_runtime(tmp_path, get_device, set_device, get_stream):
    """A module of its own (its state is the loaded file's) over another CUDA runtime; returns a call of no tokens."""
    import ctypes
    import importlib.util
    import shutil
    import tempfile

    pkg_build.build()
    path = shutil.copy(pkg_build.NATIVE, tempfile.mkdtemp(dir=tmp_path))  # (a loaded file is not written over)
    spec = importlib.util.spec_from_file_location("_native", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    L = pk.library()
    m.setup(torch.float16, torch.bfloat16, torch.float8_e4m3fn, torch.int32, torch.int64, torch.float32, get_device,
            set_device, get_stream,
            *[ctypes.cast(f, ctypes.c_void_p).value for f in (L.pa_qk_norm_rope, L.pa_qk_norm_rope_write,
                                                              L.pa_decode_window, L.pa_prefill_varlen_window)])
    x = Rows(3)
    return lambda: m.qk_norm_rope(x, x, x, x, None, (None, None, None, 1e-6, 1.0, False))


def fails(*args):
    raise RuntimeError("the runtime's error")


def test_the_device_is_changed_and_put_back(tmp_path):
    at = []
    call = with_runtime(tmp_path, lambda: at[-1] if at else 0, at.append, lambda d: 1000 + d)
    assert call() == 0
    assert at == [3, 0]


@pytest.mark.parametrize("failing", ["get_device", "set_device", "get_stream"])
def test_an_error_of_the_runtime_is_the_callers(tmp_path, failing):
    """... and leaves the current device as it was."""
    at = []
    runtime = dict(get_device=lambda: at[-1] if at else 0, set_device=at.append, get_stream=lambda d: 0)
    runtime[failing] = fails
    call = with_runtime(tmp_path, **runtime)
    for _ in range(3):
        with pytest.raises(RuntimeError, match="the runtime's error"):
            call()
    assert at == [] or at[-1] == 0


def test_a_runtime_that_answers_no_number(tmp_path):
    at = []
    call = with_runtime(tmp_path, lambda: "0", at.append, lambda d: 0)
    with pytest.raises(TypeError):
        call()
    assert at == []
    call = with_runtime(tmp_path, lambda: 0, at.append, lambda d: "0")
    with pytest.raises(TypeError):
        call()
    assert at == [] or at[-1] == 0


def test_the_module_is_named_for_its_interpreter(native):
    """Another Python in the same tree must not load a module built for this one."""
    import importlib.machinery
    import os

    assert os.path.samefile(native.__file__, pkg_build.NATIVE)
    assert os.path.basename(pkg_build.NATIVE) == "_native" + importlib.machinery.EXTENSION_SUFFIXES[0]
    assert not os.path.exists(os.path.join(pkg_build.PKG, "_native.so"))

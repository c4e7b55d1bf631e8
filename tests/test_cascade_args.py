"""pa_varlen_cascade: arguments that the host refuses before any launch.  No GPU."""
import ctypes as C

import pytest

import paged_kv_cache_75_gb300 as pk
from paged_kv_cache_75_gb300 import build as pkg_build

FAKE = 1 << 20  # an aligned address that nothing dereferences


@pytest.fixture(scope="module")
def lib():
    pkg_build.build()
    return pk.library()


def call(lib, cache=None, **kw):
    c = pk._binding._Cache(FAKE, FAKE, 8, 16, 2, 128, pk.PA_F16, 1.0, 1.0)
    for k, v in (cache or {}).items():
        setattr(c, k, v)
    a = dict(out=FAKE, q=FAKE, dtype=pk.PA_F16, table=FAKE, width=4, cu_q=FAKE, cu_k=FAKE, seqs=3, total_q=9, max_q=3,
             max_k=64, heads=8, scale=0.1, cu_groups=FAKE, shared=FAKE, groups=2, max_group=2, max_shared=32, ws=FAKE,
             ws_bytes=1 << 40)
    a.update(kw)
    return lib.pa_varlen_cascade(a["out"], a["q"], a["dtype"], C.byref(c), a["table"], a["width"], a["cu_q"], a["cu_k"],
                                 a["seqs"], a["total_q"], a["max_q"], a["max_k"], a["heads"], a["scale"], a["cu_groups"],
                                 a["shared"], a["groups"], a["max_group"], a["max_shared"], a["ws"], a["ws_bytes"], None,
                                 None)


@pytest.mark.parametrize("kw,code", [
    (dict(out=None), 1), (dict(q=None), 1), (dict(table=None), 1), (dict(cu_q=None), 1), (dict(cu_k=None), 1),
    (dict(cu_groups=None), 1), (dict(shared=None), 1), (dict(ws=None), 1), (dict(ws=FAKE + 8), 1), (dict(ws_bytes=64), 1),
    (dict(out=FAKE + 8), 1), (dict(q=FAKE + 2), 1), (dict(seqs=-1), 1), (dict(groups=-1), 1), (dict(groups=0), 1),
    (dict(total_q=-1), 1), (dict(max_q=-1), 1), (dict(max_k=-1), 1), (dict(max_group=-1), 1), (dict(max_shared=-16), 1),
    (dict(max_shared=80), 1), (dict(max_shared=24), 1), (dict(scale=0.0), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(heads=7), 1), (dict(width=0), 1), (dict(heads=32), 2), (dict(dtype=pk.PA_BF16), 2),
    (dict(dtype=pk.PA_F32), 2), (dict(cache=dict(head_size=64)), 2), (dict(cache=dict(block_size=8), max_shared=32), 2),
    (dict(cache=dict(kv_dtype=pk.PA_FP8_E4M3)), 2), (dict(cache=dict(k_cache=None)), 1), (dict(seqs=6000, groups=145), 2),
    (dict(seqs=0), 0), (dict(max_q=0), 0), (dict(total_q=0), 0)])
def test_refused(lib, kw, code):
    assert call(lib, **kw) == code


def test_workspace_size(lib):
    f = pk.pa_varlen_cascade_workspace_size
    ok = (4, 64, 32, 8, 128, 16, 4096, 1024, 16)
    assert f(*ok) >= 64 * 32 * 2 * (128 + 1) * 4
    for i in (0, 1, 2, 3, 4, 5, 8):
        bad = list(ok)
        bad[i] = 0
        assert f(*bad) == 0
    assert f(4, 64, 30, 8, 128, 16, 4096, 1024, 16) == 0

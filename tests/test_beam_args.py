"""Beam selection and reordering: arguments that the host refuses before any launch.  No GPU."""
import ctypes as C

import pytest

import paged_kv_cache_75_gb300 as pk
from paged_kv_cache_75_gb300 import build as pkg_build

FAKE = 1 << 20  # an aligned address that nothing dereferences


@pytest.fixture(scope="module")
def lib():
    pkg_build.build()
    return pk.library()


def select(lib, **kw):
    a = dict(scores_out=FAKE, rows_out=FAKE, tokens_out=FAKE, logits=FAKE, dtype=pk.PA_BF16, stride=1000, vocab=1000,
             rows=4, scores=FAKE, cu=FAKE, requests=2, allowed=None, allowed_stride=32, ended=None, end_token=0, k=4,
             ws=FAKE, ws_bytes=1 << 30)
    a.update(kw)
    return lib.pa_beam_select(a["scores_out"], a["rows_out"], a["tokens_out"], a["logits"], a["dtype"], a["stride"],
                              a["vocab"], a["rows"], a["scores"], a["cu"], a["requests"], a["allowed"],
                              a["allowed_stride"], a["ended"], a["end_token"], a["k"], a["ws"], a["ws_bytes"], None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=pk.PA_FP8_E4M3), 2), (dict(dtype=9), 2), (dict(k=65), 2), (dict(vocab=(1 << 23) + 1, stride=1 << 24), 2), (dict(k=0), 1), (dict(vocab=0), 1),
    (dict(stride=999), 1), (dict(rows=-1), 1), (dict(requests=-1), 1), (dict(logits=None), 1), (dict(scores=None), 1),
    (dict(cu=None), 1), (dict(scores_out=None), 1), (dict(rows_out=None), 1), (dict(tokens_out=None), 1),
    (dict(logits=FAKE + 1), 1), (dict(logits=FAKE + 2, dtype=pk.PA_F32), 1), (dict(allowed=FAKE, allowed_stride=31), 1),
    (dict(ended=FAKE, end_token=1000), 1), (dict(ended=FAKE, end_token=-1), 1), (dict(ws=None), 1),
    (dict(ws=FAKE + 8), 1), (dict(ws_bytes=100), 1), (dict(requests=0), 0)])
def test_select(lib, kw, code):
    assert select(lib, **kw) == code


def test_workspace_size(lib):
    one = pk.pa_beam_select_workspace_size(1, 2048, 4)
    assert one >= 16 + 4 * 8 + 8
    assert pk.pa_beam_select_workspace_size(10, 20480, 64) >= 100 * (16 + 64 * 8)
    for bad in ((0, 10, 4), (4, 0, 4), (4, 10, 0), (4, 10, 65)):
        assert pk.pa_beam_select_workspace_size(*bad) == 0


def cache(**kw):
    c = pk._binding._Cache(FAKE, FAKE, 8, 16, 2, 128, pk.PA_F16, 1.0, 1.0)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def reorder(lib, caches=None, layers=None, **kw):
    caches = [cache()] if caches is None else caches
    a = dict(parents=FAKE, n=3, table=FAKE, rows=2, width=4, lens=FAKE, spare=FAKE, table_out=FAKE + 64, lens_out=FAKE + 64,
             slots=FAKE, used=FAKE)
    a.update(kw)
    arr = (pk._binding._Cache * max(len(caches), 1))(*caches)
    return lib.pa_beam_reorder(arr, len(caches) if layers is None else layers, a["parents"], a["n"], a["table"], a["rows"],
                               a["width"], a["lens"], a["spare"], a["table_out"], a["lens_out"], a["slots"], a["used"],
                               None, None)


@pytest.mark.parametrize("kw,code", [
    (dict(layers=0), 1), (dict(n=-1), 1), (dict(rows=-1), 1), (dict(width=0), 1), (dict(parents=None), 1),
    (dict(table=None), 1), (dict(lens=None), 1), (dict(spare=None), 1), (dict(table_out=None), 1), (dict(lens_out=None), 1),
    (dict(slots=None), 1), (dict(used=None), 1), (dict(table_out=FAKE), 1), (dict(lens_out=FAKE), 1), (dict(n=0), 0),
    (dict(caches=[cache(), cache(k_cache=None)]), 1), (dict(caches=[cache(), cache(block_size=32)]), 1),
    (dict(caches=[cache(), cache(num_blocks=9)]), 1), (dict(caches=[cache(), cache(kv_dtype=pk.PA_BF16)]), 1),
    (dict(caches=[cache(kv_dtype=pk.PA_F32)]), 2), (dict(caches=[cache(num_kv_heads=1 << 20, head_size=128)]), 2)])
def test_reorder(lib, kw, code):
    assert reorder(lib, **kw) == code


def test_no_caches(lib):
    assert lib.pa_beam_reorder(None, 1, FAKE, 1, FAKE, 1, 1, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, None) == 1


def test_a_binary32_cache_is_refused_everywhere(lib):
    c = cache(kv_dtype=pk.PA_F32)
    assert lib.pa_kv_cache_write(C.byref(c), FAKE, FAKE, pk.PA_F16, 1, 256, FAKE, None, None) == 2
    assert lib.pa_copy_blocks(C.byref(c), FAKE, 1, None, None) == 2
    ok = cache()
    assert lib.pa_kv_cache_write(C.byref(ok), FAKE, FAKE, pk.PA_F32, 1, 256, FAKE, None, None) == 2

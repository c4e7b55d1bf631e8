"""Workspace sizes and refusals of the windowed attention calls.  No GPU."""
import ctypes as C
import math

import pytest
import torch

import paged_kv_cache_75_gb300 as pk
import window_ref as R
from paged_kv_cache_75_gb300 import build as pkg_build

FAKE = 1 << 20  # a 16-byte aligned, never dereferenced address
MAX = 2 ** 31 - 1


@pytest.fixture(scope="module")
def lib():
    pkg_build.build()
    return pk.library()


def cache(**kw):
    c = pk._binding._Cache(FAKE, FAKE, 8, 16, 2, 128, pk.PA_F16, 1.0, 1.0)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


def test_decode_window_workspace(lib):
    size = pk.pa_decode_window_workspace_size
    # the sinks' block, the window's and the rest of its first: 16 + 481 + 15 tokens fit one partition of 512
    assert size(4, 8, 128, 100000, 16, 481, 4, 512) == 0
    rows = 4 * 8 * 2
    assert size(4, 8, 128, 100000, 16, 482, 4, 512) >= rows * 129 * 4
    # automatic: parts of 128 tokens or more
    assert size(4, 8, 128, 100000, 16, 97, 4) == 0
    assert rows * 129 * 4 <= size(4, 8, 128, 100000, 16, 98, 4) < size(4, 8, 128, 100000, 16, 2000, 4)
    assert size(4, 8, 128, 100000, 16, 2000, 4) < pk.pa_decode_workspace_size(4, 8, 128, 100000, 16)
    assert size(4, 8, 128, 300, 16, MAX, MAX, 128) == pk.pa_decode_workspace_size(4, 8, 128, 300, 16, 128)
    assert size(4, 8, 128, 300, 16, 0, 4) == 0 and size(4, 8, 128, 300, 16, 8, -1) == 0


def test_decode_window_rejects_bad_arguments_before_launch(lib):
    def call(c=None, H=4, dt=pk.PA_F16, window=8, sinks=2, P=0, ws=None, ws_bytes=0, max_len=64, scale=0.1):
        return lib.pa_decode_window(FAKE, FAKE, dt, C.byref(c or cache()), FAKE, 4, FAKE, 2, max_len, H, scale, window,
                                    sinks, P, ws, ws_bytes, None, None)
    assert call(window=0) == 1 and call(window=-5) == 1 and call(sinks=-1) == 1
    assert call(H=3) == 1 and call(scale=math.nan) == 1 and call(P=24) == 1
    assert call(dt=pk.PA_BF16) == 2 and call(c=cache(head_size=96)) == 2 and call(c=cache(block_size=8)) == 2
    assert call(window=400, max_len=5000, P=64) == 1                      # split: needs a workspace
    assert call(window=400, max_len=5000, P=64, ws=FAKE, ws_bytes=64) == 1
    assert lib.pa_decode_window(None, None, 0, C.byref(cache()), None, 4, None, 0, 64, 4, 0.1, 8, 2, 0, None, 0, None,
                                None) == 0                                # an empty batch


def test_reference_against_a_dense_softmax():
    g = torch.Generator().manual_seed(1)
    kc, vc = torch.randn(5, 2, 16, 64, generator=g), torch.randn(5, 2, 16, 64, generator=g)
    row = torch.tensor([3, 0, 4])
    q = torch.randn(40, 4, 64, generator=g)
    L, window, sinks = 45, 9, 3
    out, _ = R.attend(q, range(5, 45), L, row, kc, vc, 0.125, window, sinks)
    K = kc[row].permute(1, 0, 2, 3).reshape(2, 48, 64)[:, :L].double().repeat_interleave(2, 0)
    V = vc[row].permute(1, 0, 2, 3).reshape(2, 48, 64)[:, :L].double().repeat_interleave(2, 0)
    p, t = torch.arange(5, 45)[:, None], torch.arange(L)[None]
    seen = (t <= p) & ((t > p - window) | (t < sinks))
    want = torch.nn.functional.scaled_dot_product_attention(q.double().transpose(0, 1), K, V, seen, scale=0.125)
    assert torch.allclose(out, want.transpose(0, 1), atol=1e-12)
    full, _ = R.attend(q, range(5, 45), L, row, kc, vc, 0.125, 100, 0)
    want = torch.nn.functional.scaled_dot_product_attention(q.double().transpose(0, 1), K, V, t <= p, scale=0.125)
    assert torch.allclose(full, want.transpose(0, 1), atol=1e-12)
    assert R.seen_blocks(45, 44, 9, 3, 16).tolist() == [True, False, True]


def test_prefill_window_rejects_bad_arguments_before_launch(lib):
    def call(c=None, H=4, dt=pk.PA_F16, window=8, sinks=2, scale=0.1, n=2, max_q=8, bt=FAKE):
        return lib.pa_prefill_varlen_window(FAKE, FAKE, dt, C.byref(c or cache()), bt, 4, FAKE, FAKE, n, max_q, 64, H,
                                            scale, window, sinks, None, None)
    assert call(window=0) == 1 and call(window=-5) == 1 and call(sinks=-1) == 1
    assert call(scale=0.0) == 1 and call(scale=-0.1) == 1 and call(scale=math.nan) == 1 and call(scale=math.inf) == 1
    assert call(H=3) == 1 and call(bt=None) == 1
    assert call(dt=pk.PA_BF16) == 2 and call(c=cache(head_size=64)) == 2 and call(c=cache(block_size=8)) == 2
    assert call(c=cache(kv_dtype=pk.PA_FP8_E4M3)) == 2
    assert call(n=0) == 0 and call(max_q=0) == 0

"""Rotation frequencies (host call) against their formulas, and the refusals of pa_qk_norm_rope and
pa_qk_norm_rope_write.  No GPU."""
import ctypes as C
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_75_gb300 as pk
import rope_ref
from paged_kv_cache_75_gb300 import build as pkg_build

KINDS = [("none", {}), ("linear", dict(factor=4.0)), ("ntk", dict(factor=8.0)),
         ("yarn", dict(factor=16.0, original=8192.0)), ("yarn", dict(factor=2.0, original=100.0)),
         ("banded", dict(factor=8.0, original=8192.0))]


@pytest.fixture(scope="module")
def lib():
    pkg_build.build()
    return pk.library()


@pytest.mark.parametrize("rot", [16, 64, 128])
@pytest.mark.parametrize("base", [10000.0, 500000.0])
@pytest.mark.parametrize("kind,kw", KINDS)
def test_frequencies_follow_the_formulas(lib, rot, base, kind, kw):
    want, factor = rope_ref.theta(rot, base, kind, **kw)
    args = dict(kw)
    if "original" in args:
        args["original_max_position"] = args.pop("original")
    r = pk.rope_frequencies(rot, base, kind, device="cpu", **args)
    np.testing.assert_allclose(r.theta, want, rtol=1e-13)
    assert abs(r.factor - factor) <= 2 ** -23 * factor
    assert r.rotary_dim == rot
    turns = r.turns.numpy().view(np.uint64)
    # theta / 2 pi to 53 bits, in 2^-64 of a turn
    for t, u in zip(r.theta, turns):
        assert abs(int(u) - (t / (2 * math.pi)) % 1.0 * 2.0 ** 64) <= 2.0 ** 64 * 2.0 ** -52


def test_given_frequencies_wrap_and_keep_their_sign(lib):
    r = pk.rope_frequencies(16, scaling="given", device="cpu", theta=[0.0, 2 * math.pi, -1.0, 100.0, 1e-9, 1, 2, 3])
    u = [int(x) for x in r.turns.numpy().view(np.uint64)]
    assert u[0] == 0 and u[1] in (0, 2 ** 64 - 1)
    assert abs(u[2] - (2 ** 64 - 2 ** 64 / (2 * math.pi))) < 2 ** 13
    assert abs(u[3] - (100 / (2 * math.pi)) % 1 * 2 ** 64) < 2 ** 18


def test_frequencies_refuse_bad_arguments(lib):
    for kw in (dict(rotary_dim=0), dict(rotary_dim=15), dict(rotary_dim=16, base=1.0), dict(rotary_dim=16, base=math.nan),
               dict(rotary_dim=16, scaling="linear", factor=0.5), dict(rotary_dim=2, scaling="ntk", factor=2.0),
               dict(rotary_dim=16, scaling="yarn", factor=2.0), dict(rotary_dim=16, scaling="banded", factor=2.0),
               dict(rotary_dim=16, scaling="yarn", factor=2.0, original_max_position=100, beta_fast=1, beta_slow=2),
               dict(rotary_dim=16, scaling="banded", factor=2.0, original_max_position=100, low_freq_factor=4.0),
               dict(rotary_dim=2, scaling="given", theta=[math.inf])):
        with pytest.raises(pk.PaError):
            pk.rope_frequencies(device="cpu", **kw)
    with pytest.raises(ValueError):
        pk.rope_frequencies(16, scaling="other", device="cpu")
    with pytest.raises(ValueError):
        pk.rope_frequencies(16, scaling="given", device="cpu", theta=[1.0])
    with pytest.raises(ValueError):
        pk.rope_frequencies(16, scaling="linear", factor=2.0, device="cpu", theta=[1.0] * 8)
    f = C.c_float()
    assert lib.pa_rope_frequencies(16, 1e4, None, None, FAKE, C.byref(f)) == 1


FAKE = 1 << 20  # a 16-byte aligned, never dereferenced address


def transform(**kw):
    t = pk._binding._QKTransform(FAKE, FAKE, 1e-6, FAKE, 1.0, 64, 0)
    for k, v in kw.items():
        setattr(t, k, v)
    return t


OTHER = FAKE + (1 << 12)


def _rope(lib, tr, T=3, H=4, Hkv=2, D=128, dt=pk.PA_BF16, qs=512, ks=256, qos=512, kos=256, q=FAKE, pos=FAKE,
          k_out=OTHER, q_out=OTHER):
    return lib.pa_qk_norm_rope(q_out, k_out, q, FAKE, dt, T, H, Hkv, D, qs, ks, qos, kos, pos,
                               None if tr is None else C.byref(tr), None)


def test_rope_rejects_bad_arguments_before_launch(lib):
    ok = transform()
    assert _rope(lib, ok, T=0) == 0
    assert _rope(lib, None) == 1
    assert _rope(lib, ok, T=-1) == 1
    assert _rope(lib, ok, H=0) == 1 and _rope(lib, ok, Hkv=0) == 1
    assert _rope(lib, ok, H=5000, qs=5000 * 128, qos=5000 * 128) == 2
    assert _rope(lib, ok, D=96) == 2
    assert _rope(lib, ok, dt=pk.PA_FP8_E4M3) == 2
    assert _rope(lib, ok, qs=511) == 1 and _rope(lib, ok, ks=255) == 1
    assert _rope(lib, ok, qos=511) == 1 and _rope(lib, ok, kos=255) == 1
    assert _rope(lib, ok, q=None) == 1 and _rope(lib, ok, pos=None) == 1 and _rope(lib, ok, k_out=None) == 1
    # in place with another stride
    assert _rope(lib, ok, q_out=FAKE, qos=520) == 1 and _rope(lib, ok, k_out=FAKE, kos=264) == 1
    assert _rope(lib, transform(rotary_dim=24)) == 2
    assert _rope(lib, transform(rotary_dim=144)) == 1 and _rope(lib, transform(rotary_dim=-16)) == 1
    assert _rope(lib, transform(turns=None)) == 1 and _rope(lib, transform(turns=FAKE + 4)) == 1
    assert _rope(lib, transform(rope_factor=math.inf)) == 1
    assert _rope(lib, transform(eps=0.0)) == 1 and _rope(lib, transform(eps=math.nan)) == 1
    assert _rope(lib, transform(q_weight=FAKE + 4)) == 1 and _rope(lib, transform(k_weight=FAKE + 8)) == 1
    assert _rope(lib, transform(q_weight=None, k_weight=None, eps=0.0), T=0) == 0


def test_rope_write_rejects_bad_arguments_before_launch(lib):
    def call(tr=None, T=3, H=4, dt=pk.PA_BF16, vs=256, v=FAKE, slots=FAKE, **cache):
        c = pk._binding._Cache(FAKE, FAKE, 8, 16, 2, 128, pk.PA_BF16, 1.0, 1.0)
        for k, x in cache.items():
            setattr(c, k, x)
        tr = tr or transform()
        return lib.pa_qk_norm_rope_write(FAKE, FAKE, FAKE, v, dt, C.byref(c), T, H, 512, 256, vs, 512, FAKE, slots,
                                         C.byref(tr), None, None)

    assert call(T=0) == 0
    assert call(dt=pk.PA_F16) == 2                                # the cache has another type
    assert call(vs=255) == 1 and call(v=None) == 1 and call(slots=None) == 1
    assert call(kv_dtype=pk.PA_FP8_E4M3, k_scale=0.0) == 1
    assert call(kv_dtype=pk.PA_FP8_E4M3, v_scale=math.inf) == 1
    assert call(head_size=96) == 2 and call(k_cache=FAKE + 2) == 1 and call(block_size=0) == 1
    assert call(tr=transform(rotary_dim=8)) == 2


def test_reference_rotation_keeps_lengths_and_relative_angles():
    """The 64-bit reference itself: rotations keep a pair's length, and q . k depends on the distance alone."""
    g = torch.Generator().manual_seed(3)
    x = torch.randn(1, 1, 64, generator=g, dtype=torch.float64)
    y = torch.randn(1, 1, 64, generator=g, dtype=torch.float64)
    th, _ = rope_ref.theta(64)
    for inter in (False, True):
        a, _ = rope_ref.rows(x, [1000], th, interleaved=inter)
        b, _ = rope_ref.rows(y, [990], th, interleaved=inter)
        c, _ = rope_ref.rows(x, [70], th, interleaved=inter)
        d, _ = rope_ref.rows(y, [60], th, interleaved=inter)
        assert abs(a.norm() - x.norm()) < 1e-12
        assert abs((a * b).sum() - (c * d).sum()) < 1e-10
    n, _ = rope_ref.rows(x, [0], th, weight=torch.ones(64), eps=0.0)
    assert abs(n.pow(2).mean() - 1.0) < 1e-12


def test_turns_of_a_negative_frequency_are_as_fine(lib):
    """theta and -theta turn by the same angle the two ways at any position: a small negative frequency keeps the bits
    that a small positive one has."""
    th = [1.0, 1e-3, 1e-6, 1e-9, 1e-12, 3.7e-15, 0.25, 6.5]
    up = pk.rope_frequencies(16, scaling="given", device="cpu", theta=th).turns.numpy().view(np.uint64)
    down = pk.rope_frequencies(16, scaling="given", device="cpu", theta=[-x for x in th]).turns.numpy().view(np.uint64)
    for u, d in zip(up, down):
        assert (int(u) + int(d)) % 2 ** 64 == 0

"""Norm, rotation and cache write of query and key rows in 64 bits (CPU), written from the formulas of
include/pa_kv.h, with the error that binary32 arithmetic and one rounding may leave."""
import math

import numpy as np
import torch

# Roundings of binary32 that reach an element, in units of 2^-24 of the pair's size |a| + |b|: the angle's fraction
# to 24 bits (2^-24 of a half turn: 3.2), sincospif (2 ulp: 4) times the factor (1), the sum of squares (12 additions
# in a row or tree, halved by the root: 6), the mean and eps (2), rsqrtf (2 ulp: 4), times r and the weight (2), the
# rotation's product and fused sum (2): 24.2, counted as 32.
FP32_UNITS = 32.0


def theta(rot, base=10000.0, kind="none", factor=1.0, original=0.0, beta_fast=32.0, beta_slow=1.0, low=1.0, high=4.0):
    """(radians per position of each pair, factor of cos and sin)."""
    if kind == "ntk":
        base = base * factor ** (rot / (rot - 2))
    out = []
    for i in range(rot // 2):
        t = base ** (-2 * i / rot)
        if kind == "linear":
            t = t / factor
        elif kind == "yarn":
            def at(x):
                return rot * math.log(original / (2 * math.pi * x)) / (2 * math.log(base))
            a, b = max(0, math.floor(at(beta_fast))), min(rot - 1, math.ceil(at(beta_slow)))
            g = min(1.0, max(0.0, (i - a) / max(b - a, 0.001)))
            t = t * (1 - g) + t / factor * g
        elif kind == "banded":
            w = min(1.0, max(0.0, (original * t / (2 * math.pi) - low) / (high - low)))
            t = t * w + t / factor * (1 - w)
        out.append(t)
    return np.array(out), (0.1 * math.log(factor) + 1.0 if kind == "yarn" else 1.0)


def rows(x, positions, th, rope_factor=1.0, interleaved=False, weight=None, eps=1e-6):
    """x [T, n, D] (any type, CPU) -> (out, pair) in float64: the definition's
    rows and, for each element, |a| + |b| of the pair it comes from."""
    y = x.to(torch.float64)
    if weight is not None:
        y = y / torch.sqrt(y.pow(2).mean(-1, keepdim=True) + eps) * weight.to(torch.float64)
    out, pair = y.clone(), y.abs()
    n = len(th)
    for i in range(n):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        # the angle modulo a turn in integers: exact for any position
        turns = int(round(math.ldexp(th[i] / (2 * math.pi), 90)))
        ang = [2 * math.pi * math.ldexp((int(p) * turns) % (1 << 90), -90) for p in positions]
        co = rope_factor * torch.tensor([math.cos(v) for v in ang], dtype=torch.float64)[:, None]
        si = rope_factor * torch.tensor([math.sin(v) for v in ang], dtype=torch.float64)[:, None]
        out[..., a] = y[..., a] * co - y[..., b] * si
        out[..., b] = y[..., b] * co + y[..., a] * si
        pair[..., a] = pair[..., b] = abs(rope_factor) * (y[..., a].abs() + y[..., b].abs())
    return out, pair


def check(got, ref, pair, dtype, what=""):
    """got (CPU tensor of dtype) against ref: half a step of the type, plus binary32's part."""
    fi = torch.finfo(dtype)
    g = got.to(torch.float64)
    ref = ref.clamp(fi.min, fi.max) if dtype == torch.float8_e4m3fn else ref
    lim = ref.abs() * (fi.eps / 2) * (1 + 1e-6) + pair * FP32_UNITS * 2.0 ** -24 * (1 + fi.eps) + \
        fi.smallest_normal * fi.eps / 2
    bad = ~((g - ref).abs() <= lim)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError("%s: %d of %d off, first at %s: got %r want %r (limit %.3g)"
                             % (what, int(bad.sum()), bad.numel(), i, g[i].item(), ref[i].item(), lim[i].item()))

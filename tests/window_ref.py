"""Attention with a sliding window and sinks over a paged cache in 64 bits (CPU), from its definition, and how far
a kernel may be from it."""
import torch

# What a kernel's arithmetic leaves, relative to the absolute weighted sum of the values: a weight rounded to 11 bits
# (fp16 weights on the tensor cores; bf16 ones go in as two parts, 16 bits) is off by 2^-11; binary32 scores of a few
# units off by some 10^-5, and sums of up to thousands of terms taken 16 at a time by as much: 2^-14 together.
WEIGHTS = 2.0 ** -11 + 2.0 ** -14


def keys_of(cache, row, positions):
    """[n, Hkv, D] in float64 of a sequence's positions."""
    bs = cache.shape[2]
    blk = row[positions // bs].long()
    assert bool((blk >= 0).all())
    bits = cache.view(torch.uint8 if cache.element_size() == 1 else torch.int16) if cache.element_size() < 4 else cache
    return bits[blk, :, positions % bs].view(cache.dtype).to(torch.float64)


def attend(q, positions, L, row, k_cache, v_cache, scale, window, sinks, k_scale=1.0, v_scale=1.0):
    """Queries q [n, H, D] at `positions` of a sequence of L keys: (out, sum of
    weight * |value|), both [n, H, D] in float64."""
    n, H, D = q.shape
    Hkv = k_cache.shape[1]
    out = torch.zeros(n, H, D, dtype=torch.float64)
    mag = torch.zeros(n, H, D, dtype=torch.float64)
    for i in range(n):
        p = int(positions[i])
        t = torch.arange(L)
        t = t[(t <= p) & ((p - t < window) | (t < sinks))]
        if t.numel() == 0:
            continue
        K, V = keys_of(k_cache, row, t) * k_scale, keys_of(v_cache, row, t) * v_scale
        for h in range(H):
            g = h // (H // Hkv)
            w = torch.softmax(scale * (K[:, g] @ q[i, h].to(torch.float64)), 0)
            out[i, h] = w @ V[:, g]
            mag[i, h] = w @ V[:, g].abs()
    return out, mag


def check(got, ref, mag, what=""):
    fi = torch.finfo(got.dtype)
    g = got.cpu().to(torch.float64)
    lim = ref.abs() * (fi.eps / 2) + mag * WEIGHTS * (1 + fi.eps) + fi.smallest_normal * fi.eps / 2
    bad = ~((g - ref).abs() <= lim)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError("%s: %d of %d off, first at %s: got %r want %r (limit %.3g)"
                             % (what, int(bad.sum()), bad.numel(), i, g[i].item(), ref[i].item(), lim[i].item()))


def seen_blocks(L, first, window, sinks, bs):
    """Which blocks of a sequence of L keys hold a position that a query from position `first` on sees."""
    j = torch.arange((L + bs - 1) // bs)
    return (j * bs < min(sinks, L)) | ((j + 1) * bs > max(0, first - window + 1))

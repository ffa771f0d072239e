"""Reference of the 4-bit cache, in numpy: the codes and scales of a group of 64 channels by the definition's fp32 steps, the
values that they stand for in float64, and reads by a block table.

    m = min x, down to bf16;   s = (max x - m) / 15, up to bf16;   code = (x - m) / s to the nearest integer, cut to 0 .. 15;
    value = m + code s.  A group with something not finite, or out of range, has s = 0, m = NaN; s = 0 has codes 0.
"""
import numpy as np

GROUP = 64
F = np.float32


def bf16_toward(x, up):
    """The bf16 number (as fp32) next to x on its upper or lower side, or x."""
    x = np.ascontiguousarray(x, F)
    bits = x.view(np.uint32)
    cut = bits & np.uint32(0xFFFF0000)                      # towards zero
    more = (bits != cut) & ((x > 0) == up) & ~np.isnan(x)
    return np.where(more, cut + np.uint32(0x10000), cut).astype(np.uint32).view(F)


def quantize(x):
    """x [..., d] fp32.  Returns (codes uint8 [..., d], s and m fp32 [..., d / 64])."""
    x = np.asarray(x, F)
    y = x.reshape(*x.shape[:-1], -1, GROUP)
    with np.errstate(all="ignore"):
        lo, hi = y.min(-1), y.max(-1)
        m = bf16_toward(lo, False)
        width = (hi - m).astype(F)
        s = bf16_toward((width / F(15)).astype(F), True)
        fine = np.isfinite(y).all(-1) & np.isfinite(m) & np.isfinite(width) & np.isfinite(s)
        steps = ((y - m[..., None]).astype(F) / s[..., None]).astype(F)
        codes = np.clip(np.rint(steps), 0, 15)
    codes = np.where((fine & (s > 0))[..., None], codes, 0).astype(np.uint8).reshape(x.shape)
    return codes, np.where(fine, s, F(0)), np.where(fine, m, F(np.nan))


def values(codes, s, m):
    """In float64."""
    wide = [np.repeat(np.asarray(t, np.float64), GROUP, -1) for t in (s, m)]
    return wide[1] + codes * wide[0]


def packed(codes):
    return (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)


def unpacked(bytes_):
    out = np.empty((*bytes_.shape[:-1], 2 * bytes_.shape[-1]), np.uint8)
    out[..., 0::2], out[..., 1::2] = bytes_ & 15, bytes_ >> 4
    return out

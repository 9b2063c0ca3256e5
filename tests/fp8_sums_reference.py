"""Value-by-value bounds of the 8-bit floating-point products with fp32 sums and of what is quantized
from them, in 64 bits with numpy (no GPU, no code of the package).  Intervals: a value that was rounded may
be any that the interval before the rounding rounds to, so a value that is not next to a border of the rounding
is known exactly."""
import numpy as np

import fp8_reference as ref


def bf16(t):
    """t rounded to nearest even among bf16's normal numbers."""
    m, x = np.frexp(t)
    return np.ldexp(np.rint(m * 256), x - 8)


def fp32_sums(v, w):
    """(v w^T, how far fp32 sums may be from it) of quantized rows and a matrix.

    An instruction takes columns 8 s .. 8 s + 7 and 32 + 8 s .. of a step of 64.  The products are exact (eight
    significant bits).  Of eight that are added together each is cut below 2^-24 of the power of two of the largest,
    which itself loses nothing: 7 * 2^-24 of it.  The two eights' sums and the two steps that join them with the sum so
    far are fp32 numbers, each within 2^-24 of its size: the eights themselves, at most the sum before and one eight, and
    the sum behind.  Twice that, as the sums so far are off themselves by what has been lost."""
    M, K = v.shape
    pad = -K % 64
    v, w = np.pad(v, ((0, 0), (0, pad))), np.pad(w, ((0, 0), (0, pad)))
    total, err = np.zeros((M, w.shape[0])), np.zeros((M, w.shape[0]))
    for at in range(0, K + pad, 64):
        for s in range(4):
            before, sizes = np.abs(total), 0.0
            for lo in (at + 8 * s, at + 32 + 8 * s):
                a, b = v[:, lo:lo + 8], w[:, lo:lo + 8]
                top = np.max(np.abs(a), axis=1)[:, None] * np.max(np.abs(b), axis=1)     # the largest product is no larger
                part = a @ b.T
                total = total + part
                err += 7 * 2.0 ** -24 * top
                sizes = sizes + np.abs(part)
            err += 2.0 ** -23 * (before + np.abs(total) + 2 * sizes)
    return total, err


def quant_interval(lo, hi, halves=1):
    """(quant of the middle, how far quant of values in [lo, hi] may be from it), elementwise for rows of bf16 values."""
    mid = quant_ends(lo, hi, halves)
    center = mid[0]
    return center, np.maximum(*(np.max(np.abs(e - center), axis=0) for e in (mid[:2], mid[2:])))


def quant_ends(lo, hi, halves):
    """Both ends in the unit of the block's least and of its greatest possible largest value (roundings are monotonic)."""
    out = np.zeros((4,) + lo.shape)
    for b in ref.spans(lo.shape[1], halves):
        l, h = lo[:, b], hi[:, b]
        least = np.where((l <= 0) & (h >= 0), 0, np.minimum(np.abs(l), np.abs(h)))
        for i, top in enumerate((least, np.maximum(np.abs(l), np.abs(h)))):
            u = ref.unit(np.max(top, axis=1, keepdims=True))
            for j, e in enumerate((l, h)):
                out[2 * i + j][:, b] = ref.e4m3(np.clip(e / u, -448, 448)) * u
    return out


def cut_sums(v, w):
    """The sums of the scaled instruction as fp8_reference.product describes them, for comparison."""
    got = np.zeros((v.shape[0], w.shape[0]))
    for g in range(0, v.shape[1], 8):
        a, b = v[:, g:g + 8], w[:, g:g + 8]
        t = a[:, None, :] * b[None, :, :]
        with np.errstate(divide="ignore", invalid="ignore"):
            e = np.floor(np.log2(np.abs(a)))[:, None, :] + np.floor(np.log2(np.abs(b)))[None, :, :]
            unit = np.exp2(np.max(np.where(t != 0, e, -np.inf), axis=2, keepdims=True) - 13)
            got += np.nan_to_num(np.trunc(t / unit) * unit).sum(2)
    return got

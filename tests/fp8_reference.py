"""The block-scaled 8-bit products by their definition, in 64 bits with numpy
(no GPU, no code of the package)."""
import numpy as np

BLOCK = 128
SLOPE = {"swiglu": 1.0, "qgeglu": 1.702}


def unit(top):
    """2^c for the largest |v| of blocks: the least power of two, c >= -126, with top <= 448 * 2^c (1 for zero)."""
    m, x = np.frexp(np.where(np.isfinite(top) & (top > 0), top, 1.0))     # top = m 2^x, 1/2 <= m < 1
    c = np.maximum(x - 9 + (m > 0.875), -126)
    return np.where(np.isfinite(top), np.ldexp(1.0, np.where(top > 0, c, -126)), 1.0)


def e4m3(t):
    """t rounded to nearest even among the e4m3 values (|t| <= 448; NaN stays)."""
    with np.errstate(divide="ignore", invalid="ignore"):
        x = np.floor(np.log2(np.abs(t)))
    step = np.exp2(np.where(np.isfinite(x), np.maximum(x, -6), -6) - 3)
    return np.rint(t / step) * step


def spans(n, halves=1):
    """The blocks of a dimension as slices."""
    each = n // halves
    return [slice(h * each + lo, h * each + min(lo + BLOCK, each)) for h in range(halves) for lo in range(0, each, BLOCK)]


def quant(v, halves=1):
    """What rows stand for after quantization."""
    out = np.empty_like(v, dtype=np.float64)
    for b in spans(v.shape[1], halves):
        with np.errstate(invalid="ignore"):
            top = np.max(np.abs(v[:, b]), axis=1, keepdims=True)      # NaN stays NaN
            s = unit(top)
            out[:, b] = np.where(np.isfinite(top), e4m3(v[:, b] / s) * s, np.nan)
    return out


def quant_weights(w, halves=1):
    """(q, byte of the scale of each block) of one matrix."""
    q, s = np.empty_like(w, dtype=np.float64), []
    for r in spans(w.shape[0], halves):
        for c in spans(w.shape[1]):
            u = float(unit(np.max(np.abs(w[r, c]))))
            q[r, c] = e4m3(w[r, c] / u)
            s.append(int(np.log2(u)) + 127)
    return q, np.asarray(s, np.uint8).reshape(-1, len(spans(w.shape[1])))


def dequant(q, s, halves=1):
    """The matrix that q and the scale bytes stand for."""
    w = np.array(q, dtype=np.float64)
    for i, r in enumerate(spans(w.shape[0], halves)):
        for j, c in enumerate(spans(w.shape[1])):
            w[r, c] *= 2.0 ** (int(s[i, j]) - 127)
    return w


def act(h, slope):
    g, u = np.split(h, 2, axis=1)
    return g / (1 + np.exp(-slope * g)) * u


def act_grad(h, da, slope):
    g, u = np.split(h, 2, axis=1)
    s = 1 / (1 + np.exp(-slope * g))
    return np.concatenate([da * u * s * (1 + slope * g * (1 - s)), da * g * s], axis=1)


def product(v, w):
    """(v w^T, how far the instruction's sums may be from it) of quantized rows and a matrix.

    The matrix instruction adds products of eight neighbours (exact: eight significant bits) after cutting each below
    2^-13 of the power of two of the largest's factors, at most 2^-13 of the largest product, which itself loses
    nothing: 7 * 2^-13 of it.  All else is K fp32 additions, each within a unit in the last place of a sum that no
    sum of sizes passes: 2^-23 of it, with one block of padding."""
    a, b = np.abs(v), np.abs(w)
    lost = np.zeros((v.shape[0], w.shape[0]))
    for g in range(0, v.shape[1], 8):
        top = np.zeros_like(lost)
        for k in range(g, g + 8):
            np.maximum(top, a[:, k, None] * b[None, :, k], out=top)
        lost += top
    return v @ w.T, 7 * 2.0 ** -13 * lost + (v.shape[1] + BLOCK) * 2.0 ** -23 * (a @ b.T)


def bound(want, err):
    """How far a bf16 result may be: the sum's error, then one rounding (2^-8 of the result)."""
    return err + 2.0 ** -8 * (np.abs(want) + err) + 1e-38

"""The bounds of fp8_sums_reference on the CPU: values inside them, and the cut sums outside."""
import numpy as np

import fp8_reference as ref
import fp8_sums_reference as sums


def _case(seed, M=24, K=768, N=40):
    r = np.random.RandomState(seed)
    v = ref.quant(r.randn(M, K) * np.exp(0.5 * r.randn(M, 1)) * np.exp(0.5 * r.randn(K)))
    q, s = ref.quant_weights(r.randn(N, K) * 0.02)
    return v, ref.dequant(q, s)


def test_bf16_is_nearest_even():
    assert sums.bf16(np.array([1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, -(1 + 2.0 ** -8 + 2.0 ** -30), 0.0, 255.5])).tolist() == [
        1, 1 + 2.0 ** -6, -(1 + 2.0 ** -7), 0, 256]


def test_fp32_sums_lie_within_the_bound_and_cut_sums_do_not():
    v, w = _case(1)
    want, err = sums.fp32_sums(v, w)
    assert np.allclose(want, v @ w.T, rtol=1e-12, atol=1e-12)
    got = np.zeros(want.shape, np.float32)
    for k in range(0, v.shape[1], 8):       # another order of the same sums, every step rounded to fp32
        got = (got + (v[:, k:k + 8] @ w[:, k:k + 8].T).astype(np.float32)).astype(np.float32)
    assert np.all(np.abs(got - want) <= 2 * err)
    assert np.mean(np.abs(sums.cut_sums(v, w) - want) > err) > 0.2      # the bound tells the two apart
    # and so do their bf16 roundings: most values are known exactly, and the cut sums miss some of them
    lo, hi = sums.bf16(want - err), sums.bf16(want + err)
    assert np.mean(lo != hi) < 0.05
    cut = sums.bf16(sums.cut_sums(v, w))
    assert np.any((cut < lo) | (cut > hi))


def test_quantized_intervals_hold_what_lies_in_them():
    r = np.random.RandomState(2)
    v = sums.bf16(r.randn(50, 304))
    lo, hi = sums.bf16(v - 2.0 ** -9 * np.abs(v)), sums.bf16(v + 2.0 ** -9 * np.abs(v))
    assert np.all(sums.quant_interval(v, v, 2)[1] == 0) and np.array_equal(sums.quant_interval(v, v, 2)[0], ref.quant(v, 2))
    center, dev = sums.quant_interval(lo, hi, 2)
    for _ in range(20):
        t = np.where(r.rand(*v.shape) < 0.5, lo, hi)
        assert np.all(np.abs(ref.quant(t, 2) - center) <= dev)
    assert np.mean(dev > 0) < 0.3

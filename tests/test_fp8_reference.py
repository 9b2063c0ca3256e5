"""The reference of the 8-bit floating-point products against torch's own conversion (CPU)."""
import numpy as np
import torch

import fp8_reference as ref


def test_e4m3_is_torchs_conversion():
    t = np.concatenate([np.linspace(-448, 448, 20011), np.linspace(-0.05, 0.05, 20011),
                        np.arange(-64, 65) * 2.0 ** -10])           # with every tie among the subnormal values
    want = torch.from_numpy(t.astype(np.float32)).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(ref.e4m3(t.astype(np.float32).astype(np.float64)), want)


def test_units():
    assert ref.unit(np.array([448.0, 448.5, 449.0, 224.0, 224.5, 0.0, 1.75, 1.76])).tolist() == [
        1, 2, 2, 0.5, 1, 2.0 ** -126, 2.0 ** -8, 2.0 ** -7]
    assert ref.unit(np.array([2.0 ** -133]))[0] == 2.0 ** -126 and ref.unit(np.array([3.3e38]))[0] == 2.0 ** 120


def test_blocks_start_anew_at_the_second_half():
    assert [(s.start, s.stop) for s in ref.spans(304, 2)] == [(0, 128), (128, 152), (152, 280), (280, 304)]
    assert [(s.start, s.stop) for s in ref.spans(128)] == [(0, 128)]


def test_derivative_against_differences():
    """The derivative that dH1 is held to, against central differences of the activation."""
    r = np.random.RandomState(3)
    h, da, eps = r.randn(40, 24) * 3, r.randn(40, 12), 1e-6
    for slope in ref.SLOPE.values():
        want = np.empty_like(h)
        for j in range(h.shape[1]):
            up, down = h.copy(), h.copy()
            up[:, j] += eps
            down[:, j] -= eps
            want[:, j] = np.sum((ref.act(up, slope) - ref.act(down, slope)) * da, axis=1) / (2 * eps)
        # differences of second order: eps^2 times a third derivative below 10 * |values|, and 2^-53 / eps of rounding
        assert np.max(np.abs(ref.act_grad(h, da, slope) - want)) < 1e-7


def test_product_bound_holds_for_the_cut_it_describes():
    """Products of eight neighbours cut below 2^-13 of the largest's power of two, then joined: within the bound."""
    r = np.random.RandomState(4)
    v, w = ref.quant(r.randn(6, 264) * np.exp(r.randn(264))), ref.quant(r.randn(5, 264))
    want, err = ref.product(v, w)
    got = np.zeros_like(want)
    for g in range(0, 264, 8):
        t = v[:, None, g:g + 8] * w[None, :, g:g + 8]
        with np.errstate(divide="ignore"):
            e = np.floor(np.log2(np.abs(v[:, None, g:g + 8]))) + np.floor(np.log2(np.abs(w[None, :, g:g + 8])))
        unit = np.exp2(np.max(np.where(t != 0, e, -np.inf), axis=2, keepdims=True) - 13)
        with np.errstate(invalid="ignore"):
            got += np.nan_to_num(np.trunc(t / unit) * unit).sum(2)
    assert np.all(np.abs(got - want) <= err) and np.any(np.abs(got - want) > err / 100)

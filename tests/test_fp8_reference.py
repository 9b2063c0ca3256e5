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

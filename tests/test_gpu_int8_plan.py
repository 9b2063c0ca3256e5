"""GPU: small tiles that are many more than the CUs, so that a workgroup goes
on from tile to tile, with rows that stream beside them; the checks against 64 bits of
tests/test_gpu_int8.py."""
import pytest
import torch

from test_gpu_int8 import test_dgrad as _dgrad
from test_gpu_int8 import test_forward as _forward

pytestmark = pytest.mark.gpu

# counts, summed dimension, output columns: fewer large tiles than CUs; more, at about 100 rows an expert, where small ones
# stay; the same with one stage of the sum and with partial tiles only
CASES = [
    ([100, 64, 128, 256, 0, 65, 200, 7], 264, 11016),
    ([100, 90, 128, 70, 64, 127, 120, 101], 264, 21768),
    ([100, 90, 110, 70, 64, 127, 120, 101], 72, 21768),
]


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("act", [None, "swiglu"])
def test_forward_many_small_tiles(case, act):
    counts, K, N = CASES[case]
    _forward(counts, K, N, 1, 2, act)


@pytest.mark.parametrize("case", range(len(CASES)))
@pytest.mark.parametrize("act", [None, "qgeglu"])
def test_dgrad_many_small_tiles(case, act):
    counts, N, K = CASES[case]
    _dgrad(counts, K, N, 1, 2, act)

"""GPU: the 8-bit products at the sizes where the launches change: enough rows
and columns for large tiles (with remainders that stream and partial tiles),
rows of few-row experts that LDS holds 96, 64 or 32 of, and none; the same
checks against 64 bits as tests/test_gpu_int8.py."""
import pytest
import torch

from test_gpu_int8 import test_dgrad as _dgrad
from test_gpu_int8 import test_forward as _forward

pytestmark = pytest.mark.gpu

# counts, summed dimension, output columns, rows before and after the experts
CASES = [
    ([300, 0, 256, 511, 352, 353], 264, 11016, 3, 2),      # large tiles: 44 and 96 rows left, 255 and 97 in partial ones
    ([2049, 1, 1023], 72, 5640, 0, 0),                     # one summed stage; a single row left
    ([64, 33, 1, 130, 0, 65], 2040, 136, 0, 1),            # 64 rows of an expert in LDS
    ([64, 33, 1, 130, 0, 65], 4096, 72, 2, 0),             # 32 rows
    ([70, 3, 0, 64, 65], 4232, 136, 0, 0),                 # none: streamed rows have a launch of their own
]


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("K,N", [(c[1], c[2]) for c in CASES])
@pytest.mark.parametrize("act", [None, "swiglu"])
def test_forward_sizes(K, N, act):
    counts, _, _, lead, tail = next(c for c in CASES if c[1:3] == (K, N))
    _forward(counts, K, N, lead, tail, act)


@pytest.mark.parametrize("K,N", [(c[1], c[2]) for c in CASES])
@pytest.mark.parametrize("act", [None, "qgeglu"])
def test_dgrad_sizes(K, N, act):
    # here the output columns are K's and the sum is over N's
    counts, _, _, lead, tail = next(c for c in CASES if c[1:3] == (K, N))
    _dgrad(counts, N, K, lead, tail, act)


def test_large_tiles_of_wide_sums():
    """Large tiles, and what they leave (76 and 4 rows) in a launch of its own: LDS holds too few rows of the sum."""
    _forward([1100, 1240, 260], 2056, 6416, 0, 0, None)

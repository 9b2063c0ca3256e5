"""GPU: how many bits of du reach da, where the sums behind it add nothing of
their own: each row of dy has one value, so du = scale dy b is one product,
exact in 16 bits and rounded once by the scale (2^-24), and few rows meet in da.

The bound of da, from the formulas (e = 2^-24): du's rounding e and its three bf16
parts, which leave (2^-8)^3 = e of it; then m rows' products and the running sum of the
first part, m + 1 additions of up to 2 e each (the matrix instruction may cut where it
does not round), and as many, 2^-8 and 2^-16 as large, for the other parts, below e together
for these few rows: (2 (m + 1) + 3) e of sum|du x| in all.  Two parts would leave up to 2^-17 of du: the test makes that sum
itself and sees that the bound excludes it."""
import numpy as np
import pytest
import torch

from gpu_harness import log
from test_gpu_adapter import DEV, Problem, _f64, _gg, _within

pytestmark = pytest.mark.gpu

EPS = 2.0 ** -24


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _bf16(v):
    return torch.from_numpy(v).to(torch.bfloat16).double().numpy()


@pytest.mark.parametrize("counts,K,N,r", [([1, 1, 0, 2, 3], 264, 40, 16), ([1, 2], 520, 1032, 24), ([1, 0, 3], 136, 264, 64),
                                          ([1], 8, 8, 1)])
def test_da_keeps_three_parts_of_du(counts, K, N, r):
    gg = _gg()
    log(f"[adapter] parts {counts} K={K} N={N} r={r}")
    scale = float(np.float32(0.7123456))
    p = Problem(counts, K, N, r, seed=5 * K + N + r)
    rng = np.random.default_rng(r)
    dy = torch.zeros_like(p.dy)
    for row in range(p.M):
        n = int(rng.integers(N))
        dy[row, n] = p.dy[row, n]
    _, da, _ = gg.gg_adapter_backward(dy.to(DEV), p.dev["x"], p.dev["u"], p.offd, p.dev["a"], p.dev["b"], scale)
    x, b, dy, da = _f64(p.x), _f64(p.b), _f64(dy), _f64(da)
    missed = 0
    for e, lo, hi in p.segments():
        m = hi - lo
        if m == 0:
            continue
        du = scale * dy[lo:hi] @ b[e]
        bound = (2 * (m + 1) + 3) * EPS * (np.abs(du).T @ np.abs(x[lo:hi]))
        _within("da", da[e], du.T @ x[lo:hi], bound)
        first = _bf16(du)
        two = first + _bf16(du - first)
        missed += int(np.sum(np.abs(two.T @ x[lo:hi] - du.T @ x[lo:hi]) > bound))
    assert missed > 0, "the bound would not see a du of two parts"

"""GPU: an infinity in dy, as an overflowing loss scale makes it, reaches the
gradients as the formula says: infinite where it is infinite there, and only
there (the ranks and columns that only pad the kernels' tiles add no NaN)."""
import numpy as np
import pytest
import torch

from gpu_harness import log
from test_gpu_adapter import DEV, Problem, _f64, _gg

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("counts,K,N,r", [([3, 0, 2], 72, 40, 1), ([40, 33], 264, 136, 5), ([33, 4], 136, 264, 16),
                                          ([300, 1], 72, 40, 24), ([70], 520, 1032, 49), ([5], 64, 64, 64)])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
def test_infinite_dy(counts, K, N, r, value):
    gg = _gg()
    log(f"[adapter] {value} in dy, {counts} K={K} N={N} r={r}")
    p = Problem(counts, K, N, r, seed=K + r)
    # positive values: the formula's sums then hold infinities of one sign
    x, a, b, u = (t.abs() + 0.125 for t in (p.x, p.a, p.b, p.u))
    dy = p.dy.clone()
    row = int(p.off[1]) - 1                    # the last row of the first expert
    dy[row, N // 2] = value
    dev = [t.to(torch.bfloat16).to(DEV) for t in (dy, x, u)]
    dx, da, db = gg.gg_adapter_backward(*dev, p.offd, a.to(torch.bfloat16).to(DEV), b.to(torch.bfloat16).to(DEV), 0.5,
                                        base=p.dev["xbase"])
    torch.cuda.synchronize()
    for e, lo, hi in p.segments():
        if lo == hi:
            continue
        d = dy[lo:hi].double().numpy()
        with np.errstate(invalid="ignore"):
            du = 0.5 * d @ _f64(b[e])
        for name, got, want in (("dx", dx[lo:hi], _f64(p.xbase[lo:hi]) + du @ _f64(a[e])),
                                ("da", da[e], du.T @ _f64(x[lo:hi])), ("db", db[e], 0.5 * d.T @ _f64(u[lo:hi]))):
            got = _f64(got)
            finite = np.isfinite(want)
            assert np.array_equal(np.isfinite(got), finite), name
            assert np.array_equal(got[~finite], want[~finite], equal_nan=True), name

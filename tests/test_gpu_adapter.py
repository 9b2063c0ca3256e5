"""GPU: the expert adapters (gg_adapter_forward, gg_adapter_backward) against
their formulas in 64 bits on the CPU, and the gradients against differences.

Tolerances, from the formulas (u8 = 2^-8 is bf16's rounding, e = 2^-24 fp32's;
a sum of n products has an error of at most (n + 64) e times the sum of their
magnitudes, the 64 for its splits and scalings):
  u   u8 |u| + (K + 64) e sum|x a|
  y   from the returned u: u8 |y| + (r + 64) e (|base| + scale sum|u b|)
  dx  u8 |dx| + sum_r (u8 |du| + D) |a| with D = (N + 64) e scale sum|dy b|
      the sums' error of du, and (r + 64) e of the second sum
  da  sum_rows (u8^2 |du| + D) |x| + (rows + 64) e sum|du x|
  db  (rows + 64) e scale sum|dy u|
"""
import numpy as np
import pytest
import torch

from gpu_harness import bitwise_equal, log

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
U8, EPS = 2.0 ** -8, 2.0 ** -24
SCALE = 0.75


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _gg():
    import moe_expert_grouped_ragged_amd as gg
    return gg


def _f64(t):
    return t.detach().cpu().double().numpy()


def _normal(shape, std, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16)


def _within(name, got, want, bound):
    err = np.abs(got - want)
    assert np.all(np.isfinite(got)), name
    assert np.all(err <= bound + 1e-37), f"{name}: worst {np.max(err / (bound + 1e-37)):.3f} of the bound"


class Problem:
    def __init__(self, counts, K, N, r, lead=0, tail=0, seed=1):
        self.E, self.K, self.N, self.r = len(counts), K, N, r
        self.off = np.concatenate([[lead], lead + np.cumsum(counts)]).astype(np.int64)
        self.M = M = int(self.off[-1]) + tail
        self.lead, self.tail = lead, tail
        self.x, self.dy = _normal((M, K), 1, seed), _normal((M, N), 1, seed + 1)
        self.ybase, self.xbase = _normal((M, N), 1, seed + 2), _normal((M, K), 1, seed + 3)
        self.a, self.b = _normal((self.E, r, K), K ** -0.5, seed + 4), _normal((self.E, N, r), r ** -0.5, seed + 5)
        self.u = _normal((M, r), 1, seed + 6)
        for t in (self.x, self.dy, self.u, self.ybase, self.xbase):   # rows without an expert reach no result
            t[:lead] = float("nan")
            t[M - tail:] = float("nan")
        self.offd = torch.from_numpy(self.off).to(DEV)
        self.dev = {n: getattr(self, n).to(DEV) for n in ("x", "dy", "ybase", "xbase", "a", "b", "u")}

    def segments(self):
        return [(e, int(self.off[e]), int(self.off[e + 1])) for e in range(self.E)]


CASES = [
    # counts, K, N, r, lead, tail: empty experts, blocks that end inside, ranks of every kind
    ([1], 8, 8, 1, 0, 0),
    ([0, 3, 0, 40, 1, 0], 72, 40, 5, 2, 3),
    ([65, 96, 97, 31, 32, 33], 264, 136, 16, 0, 0),
    ([300, 0, 256, 511, 17], 520, 1032, 12, 5, 7),
    ([777, 64], 1048, 2056, 32, 0, 1),
    ([129, 0, 0, 700], 648, 1160, 49, 1, 0),
    ([1, 1, 0, 1, 2], 2688, 264, 64, 1, 0),
    ([2900, 30, 0, 601], 200, 136, 64, 0, 0),
    ([2900, 30, 0, 601], 136, 1544, 24, 0, 0),
]


@pytest.mark.parametrize("counts,K,N,r,lead,tail", CASES)
def test_forward(counts, K, N, r, lead, tail):
    gg = _gg()
    log(f"[adapter] forward {counts} K={K} N={N} r={r}")
    p = Problem(counts, K, N, r, lead, tail, seed=K + N + r)
    d = p.dev
    y0 = torch.full((p.M, N), 3.0, dtype=torch.bfloat16, device=DEV)
    u0 = torch.full((p.M, r), 5.0, dtype=torch.bfloat16, device=DEV)
    y, u = gg.gg_adapter_forward(d["x"], p.offd, d["a"], d["b"], SCALE, base=d["ybase"], y=y0, u=u0)
    y1, u1 = gg.gg_adapter_forward(d["x"], p.offd, d["a"], d["b"], SCALE)
    inplace = d["ybase"].clone()
    y2, _ = gg.gg_adapter_forward(d["x"], p.offd, d["a"], d["b"], SCALE, base=inplace, y=inplace)
    torch.cuda.synchronize()
    x, a, b, base, gy, gy1, gu = (_f64(t) for t in (p.x, p.a, p.b, p.ybase, y, y1, u))
    for e, lo, hi in p.segments():
        want = x[lo:hi] @ a[e].T
        _within("u", gu[lo:hi], want, U8 * np.abs(want) + (K + 64) * EPS * (np.abs(x[lo:hi]) @ np.abs(a[e]).T))
        delta = SCALE * gu[lo:hi] @ b[e].T
        mag = (r + 64) * EPS * SCALE * (np.abs(gu[lo:hi]) @ np.abs(b[e]).T)
        _within("y", gy[lo:hi], base[lo:hi] + delta,
                U8 * np.abs(base[lo:hi] + delta) + mag + (r + 64) * EPS * np.abs(base[lo:hi]))
        _within("y without base", gy1[lo:hi], delta, U8 * np.abs(delta) + mag)
        assert bitwise_equal(u[lo:hi], u1[lo:hi]) and bitwise_equal(y[lo:hi], y2[lo:hi])
    for g, v in ((gy, 3), (gu, 5)):
        assert np.all(g[:lead] == v) and np.all(g[p.M - tail:] == v)


@pytest.mark.parametrize("counts,K,N,r,lead,tail", CASES)
def test_backward(counts, K, N, r, lead, tail):
    gg = _gg()
    log(f"[adapter] backward {counts} K={K} N={N} r={r}")
    p = Problem(counts, K, N, r, lead, tail, seed=K + N + r)
    d = p.dev
    dx0 = torch.full((p.M, K), 3.0, dtype=torch.bfloat16, device=DEV)
    args = (d["dy"], d["x"], d["u"], p.offd, d["a"], d["b"], SCALE)
    dx, da, db = gg.gg_adapter_backward(*args, base=d["xbase"], dx=dx0)
    dx1, da1, db1 = gg.gg_adapter_backward(*args)
    acc_a, acc_b = torch.full_like(da, 0.5), torch.full_like(db, -0.25)
    inplace = d["xbase"].clone()
    dx2, _, _ = gg.gg_adapter_backward(*args, base=inplace, dx=inplace, da=acc_a, db=acc_b, accumulate=True)
    torch.cuda.synchronize()
    dy, x, u, a, b, base = (_f64(t) for t in (p.dy, p.x, p.u, p.a, p.b, p.xbase))
    gx, gx1, ga, gb = (_f64(t) for t in (dx, dx1, da, db))
    assert torch.equal(da, da1) and torch.equal(db, db1)     # equal calls, equal bits
    assert torch.allclose(acc_a, da + 0.5, rtol=0, atol=2 ** -22 * (1 + float(da.abs().max())))
    assert torch.allclose(acc_b, db - 0.25, rtol=0, atol=2 ** -22 * (1 + float(db.abs().max())))
    for e, lo, hi in p.segments():
        if lo == hi:
            assert not ga[e].any() and not gb[e].any()
            assert bool((acc_a[e] == 0.5).all()) and bool((acc_b[e] == -0.25).all())
            continue
        m = hi - lo
        du = SCALE * dy[lo:hi] @ b[e]
        D = (N + 64) * EPS * SCALE * (np.abs(dy[lo:hi]) @ np.abs(b[e]))
        want = du @ a[e]
        extra = (U8 * np.abs(du) + D) @ np.abs(a[e]) + (r + 64) * EPS * (np.abs(du) @ np.abs(a[e]))
        _within("dx without base", gx1[lo:hi], want, U8 * (np.abs(want) + extra) + extra)
        full = base[lo:hi] + want
        _within("dx", gx[lo:hi], full, U8 * (np.abs(full) + extra) + extra + 64 * EPS * np.abs(base[lo:hi]))
        _within("da", ga[e], du.T @ x[lo:hi],
                (U8 * U8 * np.abs(du) + D).T @ np.abs(x[lo:hi]) + (m + 64) * EPS * (np.abs(du).T @ np.abs(x[lo:hi])))
        _within("db", gb[e], SCALE * dy[lo:hi].T @ u[lo:hi],
                (m + 64) * EPS * SCALE * (np.abs(dy[lo:hi]).T @ np.abs(u[lo:hi])))
        assert bitwise_equal(dx[lo:hi], dx2[lo:hi])
    assert np.all(gx[:lead] == 3) and np.all(gx[p.M - tail:] == 3)


@pytest.mark.parametrize("counts,K,N,r", [([40, 0, 33], 264, 136, 12), ([300], 136, 520, 33)])
def test_gradients_against_differences(counts, K, N, r):
    """y is linear in x, a and b alone, so a difference of any step is a
    derivative: with dy the difference itself, sum dy (y1 - y0) = <gradient,
    step>.  The bound is bf16's rounding of y0, y1 and of u behind them."""
    gg = _gg()
    p = Problem(counts, K, N, r, seed=77)
    d = p.dev
    y0, u0 = gg.gg_adapter_forward(d["x"], p.offd, d["a"], d["b"], SCALE)
    for which, std in (("x", 0.5), ("a", 0.5 * K ** -0.5), ("b", 0.5 * r ** -0.5)):
        log(f"[adapter] difference in {which}")
        step = _normal(tuple(d[which].shape), std, 5).to(DEV)
        moved = dict(d)
        moved[which] = d[which] + step                     # rounded to bf16: the step that was taken
        step = moved[which].double() - d[which].double()
        y1, u1 = gg.gg_adapter_forward(moved["x"], p.offd, moved["a"], moved["b"], SCALE)
        dy = (y1.float() - y0.float()).to(torch.bfloat16)
        dx, da, db = gg.gg_adapter_backward(dy, d["x"], u0, p.offd, d["a"], d["b"], SCALE)
        grad = {"x": dx, "a": da, "b": db}[which].double()
        left = float((dy.double() * (y1.double() - y0.double())).sum())
        right = float((grad * step).sum())
        # |b| |u| bounds y's terms: u's rounding moves y by u8 of them
        mag = sum(float((dy[lo:hi].double().abs() * ((u0[lo:hi].double().abs() + u1[lo:hi].double().abs())
                         @ moved["b"][e].double().abs().t().contiguous()) * SCALE).sum()) for e, lo, hi in p.segments())
        bound = U8 * (mag + float((dy.double().abs() * (y0.double().abs() + y1.double().abs())).sum())
                      + float((grad.abs() * step.abs()).sum()))
        assert abs(left - right) <= bound, (which, left, right, bound)
        assert abs(left - right) <= 0.1 * abs(left)        # far inside: the roundings are independent


def test_bad_offsets_stay_in_bounds():
    """Decreasing and out-of-range offsets: results are undefined, but nothing
    outside the buffers is touched and the calls return."""
    gg = _gg()
    p = Problem([40, 40, 40], 72, 136, 16)
    d = p.dev
    guard = torch.full((p.M + 64, 72), 7.0, dtype=torch.bfloat16, device=DEV)
    wg = torch.full((gg.adapter_workspace_bytes(p.M, 3, 136, 72, 16) + 4096,), 9, dtype=torch.uint8, device=DEV)
    for off in ([0, 120, 0, 120], [-5, 300, 20, 10], [120, 0, 120, 0], [1 << 40, 0, 3, -(1 << 40)]):
        offd = torch.tensor(off, device=DEV)
        gg.gg_adapter_forward(d["x"], offd, d["a"], d["b"], SCALE)
        gg.gg_adapter_backward(d["dy"], d["x"], d["u"], offd, d["a"], d["b"], SCALE, dx=guard[:p.M], workspace=wg[:-4096])
        torch.cuda.synchronize()
        assert bool((guard[p.M:] == 7).all()) and bool((wg[-4096:] == 9).all())


def test_no_rows():
    gg = _gg()
    a, b = _normal((3, 8, 64), 1, 1).to(DEV), _normal((3, 40, 8), 1, 2).to(DEV)
    off = torch.zeros(4, dtype=torch.int64, device=DEV)
    e = lambda w: torch.empty(0, w, dtype=torch.bfloat16, device=DEV)   # noqa: E731
    y, u = gg.gg_adapter_forward(e(64), off, a, b, 1.0)
    assert y.shape == (0, 40) and u.shape == (0, 8)
    dx, da, db = gg.gg_adapter_backward(e(40), e(64), e(8), off, a, b, 1.0)
    assert dx.shape == (0, 64) and not da.any() and not db.any()


def test_other_stream():
    gg = _gg()
    p = Problem([65, 0, 300], 264, 296, 24)
    d = p.dev
    args = (d["dy"], d["x"], d["u"], p.offd, d["a"], d["b"], SCALE)
    want = gg.gg_adapter_backward(*args)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    got = gg.gg_adapter_backward(*args, stream=st)
    st.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_binding_refuses():
    gg = _gg()
    p = Problem([2, 2], 64, 48, 8)
    d = p.dev
    x, off, a, b = d["x"], p.offd, d["a"], d["b"]
    big = torch.empty(2, 65, 64, dtype=torch.bfloat16, device=DEV), torch.empty(2, 48, 65, dtype=torch.bfloat16, device=DEV)
    bwd = lambda **kw: gg.gg_adapter_backward(d["dy"], x, d["u"], off, a, b, 1.0, **kw)   # noqa: E731
    for i, call in enumerate([
            lambda: gg.gg_adapter_forward(x.float(), off, a, b, 1.0),
            lambda: gg.gg_adapter_forward(x, off, a.float(), b, 1.0),
            lambda: gg.gg_adapter_forward(x, off, a, b[:1], 1.0),
            lambda: gg.gg_adapter_forward(x, off, a, b[:, :, :4].contiguous(), 1.0),
            lambda: gg.gg_adapter_forward(x[:, :32].contiguous(), off, a, b, 1.0),
            lambda: gg.gg_adapter_forward(x, off[:2], a, b, 1.0),
            lambda: gg.gg_adapter_forward(x, off, *big, 1.0),
            lambda: gg.gg_adapter_forward(x, off, a, b, 1.0, base=x),
            lambda: gg.gg_adapter_forward(x.t().contiguous().t(), off, a, b, 1.0),
            lambda: bwd(base=d["dy"]),
            lambda: bwd(accumulate=True),
            lambda: bwd(da=torch.empty(2, 8, 64, dtype=torch.bfloat16, device=DEV)),
            lambda: bwd(workspace=torch.empty(4, device=DEV)),
    ]):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was accepted")

"""GPU: the 8-bit expert products (gg_int8_quantize_rows, gg_int8_pack,
gg_int8_forward, gg_int8_dgrad) against their definition in 64 bits on the
CPU.

Tolerances, from the formulas:
  * q of bf16 rows equals the 64-bit definition exactly (127 v is exact in
    fp32 and v 127 / top is a tie or at least 1/512 away from one).
  * y and dx: the integer sum is exact; its conversion, two scalings and the
    scale itself round to fp32 (4 * 2^-24), then once to bf16 (8 bits: 2^-8).
  * scaled operands (input gradient): v = ws dy rounds to fp32, and a value
    within 127 * 4 * 2^-24 of a tie may round either way, one step of that
    row's s times the weight it meets.
  * A and dH1: the sigmoid's exp2 and reciprocal are within 2^-19 for
    |gate| <= 16, and a derivative sums two such terms; then bf16 (2^-8).
"""
import numpy as np
import pytest
import torch

from gpu_harness import bitwise_equal, log

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
SLOPE = {"swiglu": 1.0, "qgeglu": 1.702}
U = 2.0 ** -8 + 4 * 2.0 ** -24


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _gg():
    import moe_expert_grouped_ragged_amd as gg
    return gg


def _f64(t):
    return t.detach().cpu().double().numpy()


def _quant(v):
    """(q, s) of float64 rows by the definition; rows that are not finite give q = 0, s = NaN."""
    with np.errstate(invalid="ignore", divide="ignore"):
        top = np.max(np.abs(v), axis=1, keepdims=True)
        q = np.rint(v * 127 / top)
    bad = ~np.isfinite(top[:, 0])
    q[(top[:, 0] == 0) | bad] = 0
    s = top[:, 0] / 127
    s[bad] = np.nan
    return q, s


def _close(got, want, extra=0.0, tol=U):
    got, want = np.asarray(got), np.asarray(want)
    assert np.array_equal(np.isnan(got), np.isnan(want))
    m = ~np.isnan(want)
    extra = np.broadcast_to(extra, want.shape)[m]
    err = np.abs(got[m] - want[m])
    bound = tol * (np.abs(want[m]) + extra) + extra + 1e-37   # the result that is rounded is want +- extra
    assert np.all(err <= bound), f"worst {np.max(err / bound):.3f} of the bound"


def _rows(M, K, seed, spread=0.5):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g) * torch.exp(spread * torch.randn(M, 1, generator=g))
    return x.to(torch.bfloat16)


def _weights(E, N, K, seed):
    g = torch.Generator().manual_seed(seed)
    w = (torch.randn(E * N, K, generator=g) * 0.02).to(torch.bfloat16)
    q, s = _quant(w.double().numpy())
    return torch.from_numpy(q.astype(np.int8)).view(E, N, K), torch.from_numpy(s.astype(np.float32)).view(E, N)


def _offsets(counts, lead=0):
    return np.concatenate([[lead], lead + np.cumsum(counts)]).astype(np.int64)


@pytest.mark.parametrize("M,K", [(1, 8), (3, 72), (130, 512), (65, 520), (9, 1048), (40, 4096), (5, 8200)])
def test_quantize_rows_equals_the_definition(M, K):
    gg = _gg()
    log(f"[int8] quantize M={M} K={K}")
    x = _rows(M, K, M * 1000 + K)
    x[M // 2] = 0
    if M > 2:
        x[1] *= 2.0 ** -130          # subnormal values
        x[2] *= 2.0 ** 120
        x[0, ::2] = x[0].abs().max() / 2    # 63.5 steps: ties
    q, s = gg.gg_int8_quantize_rows(x.to(DEV))
    qr, sr = _quant(x.double().numpy())
    assert np.array_equal(q.cpu().numpy(), qr)
    assert np.all(np.abs(_f64(s) - sr) <= 2.0 ** -24 * sr + 2.0 ** -150)


def test_quantize_rows_not_finite():
    gg = _gg()
    x = _rows(6, 264, 5)
    x[1, 7], x[2, 0], x[3, 263], x[4, 5], x[4, 6] = float("inf"), float("-inf"), float("nan"), float("inf"), float("nan")
    q, s = gg.gg_int8_quantize_rows(x.to(DEV))
    s, q = s.cpu(), q.cpu()
    assert torch.isnan(s[1:5]).all() and torch.isfinite(s[[0, 5]]).all()
    assert (q[1:5] == 0).all()


# counts cover empty experts, single rows, every 32-row block count of a small
# expert, and tiles with and without a remainder
CASES = [
    ([1], 8, 8, 0, 0),
    ([0, 3, 0, 40, 1, 0], 72, 40, 2, 3),
    ([65, 96, 97, 31, 32, 33], 264, 136, 0, 0),
    ([300, 0, 256, 511, 352, 353], 512, 520, 5, 7),
    ([777], 1048, 2056, 0, 1),
    ([1, 1, 0, 1, 2], 2688, 264, 1, 0),
]


def _reference_forward(v, s_q, wq, ws, off):
    y = np.full((v.shape[0], wq.shape[1]), np.nan)
    q, s = s_q
    for e in range(len(off) - 1):
        lo, hi = off[e], off[e + 1]
        y[lo:hi] = (q[lo:hi] @ wq[e].T) * s[lo:hi, None] * ws[e][None]
    return y


@pytest.mark.parametrize("counts,K,N,lead,tail", CASES)
@pytest.mark.parametrize("act", [None, "swiglu", "qgeglu"])
def test_forward(counts, K, N, lead, tail, act):
    gg = _gg()
    E, off = len(counts), _offsets(counts, lead)
    M = int(off[-1]) + tail
    log(f"[int8] forward E={E} M={M} K={K} N={N} {act}")
    x = _rows(M, K if act is None else 2 * K, 11 * M + K)
    x[:lead] = float("nan")                 # rows that no expert owns are not read into any result
    x[M - tail:] = float("nan")
    live = np.arange(off[0], off[-1])
    if len(live) > 4:
        x[live[1]] = 0                       # a padding row
        x[live[3], 5] = float("inf")         # a broken row spoils itself alone
    wq, ws = _weights(E, N, K, 7 + N)
    packed = gg.gg_int8_pack(wq.to(DEV), ws.to(DEV))
    offd = torch.from_numpy(off).to(DEV)
    y0 = torch.full((M, N), 3.0, dtype=torch.bfloat16, device=DEV)
    a0 = None if act is None else torch.full((M, K), 5.0, dtype=torch.bfloat16, device=DEV)
    y, a = gg.gg_int8_forward(x.to(DEV), offd, packed, E, N, K, activation=act, a_out=a0, y=y0.clone())
    torch.cuda.synchronize()
    if act is None:
        v = x.double().numpy()
    else:
        g, u = _f64(x[:, :K]), _f64(x[:, K:])
        with np.errstate(invalid="ignore", over="ignore"):
            want = g / (1 + np.exp(-SLOPE[act] * g)) * u
        v = _f64(a)
        fine = live[np.isfinite(want[live]).all(1) & np.isfinite(v[live]).all(1)]
        _close(v[fine], want[fine], tol=U + 2.0 ** -17)
        assert np.all(v[:lead] == 5) and np.all(v[M - tail:] == 5)
        y2, none = gg.gg_int8_forward(x.to(DEV), offd, packed, E, N, K, activation=act, y=y0.clone())
        assert none is None and torch.equal(y2.view(torch.int16), y.view(torch.int16))
    ref = _reference_forward(v, _quant(v), wq.double().numpy(), ws.double().numpy(), off)
    got = _f64(y)
    _close(got[live], ref[live])
    assert np.all(got[:lead] == 3) and np.all(got[M - tail:] == 3)


@pytest.mark.parametrize("counts,K,N,lead,tail", CASES)
@pytest.mark.parametrize("act", [None, "swiglu", "qgeglu"])
def test_dgrad(counts, K, N, lead, tail, act):
    gg = _gg()
    if act is not None and N % 16:
        N += 8
    E, off = len(counts), _offsets(counts, lead)
    M = int(off[-1]) + tail
    log(f"[int8] dgrad E={E} M={M} K={K} N={N} {act}")
    live = np.arange(off[0], off[-1])
    dy = _rows(M, N if act is None else N // 2, 13 * M + K)
    dy[:lead] = float("nan")
    dy[M - tail:] = float("nan")
    if len(live) > 4:
        dy[live[2]] = 0
        dy[live[4], 3] = float("nan")
    h1 = None if act is None else _rows(M, N, 17 * M + K)
    wq, ws = _weights(E, N, K, 9 + N)
    packed = gg.gg_int8_pack_transposed(wq.to(DEV), ws.to(DEV))
    offd = torch.from_numpy(off).to(DEV)
    dx0 = torch.full((M, K), 3.0, dtype=torch.bfloat16, device=DEV)
    d0 = None if act is None else torch.full((M, N), 5.0, dtype=torch.bfloat16, device=DEV)
    dx, dh1 = gg.gg_int8_dgrad(dy.to(DEV), offd, packed, E, N, K, h1=None if act is None else h1.to(DEV), activation=act,
                               dh1_out=d0, dx=dx0.clone())
    torch.cuda.synchronize()
    if act is None:
        g32 = dy.float().numpy()
    else:
        k, d = SLOPE[act], _f64(dy)
        gate, up = _f64(h1[:, :N // 2]), _f64(h1[:, N // 2:])
        sg = 1 / (1 + np.exp(-k * gate))
        # both terms of the derivative carry the sigmoid's error: compare against their magnitudes' sum
        want = np.concatenate([d * up * sg * (1 + k * gate * (1 - sg)), d * gate * sg], 1)
        size = np.concatenate([np.abs(d * up * sg) * (1 + np.abs(k * gate * (1 - sg))), np.abs(d * gate * sg)], 1)
        got = _f64(dh1)
        _close(got[live], want[live], extra=2.0 ** -17 * np.nan_to_num(size[live]))
        assert np.all(got[:lead] == 5) and np.all(got[M - tail:] == 5)
        g32 = dh1.float().cpu().numpy()
        dx2, none = gg.gg_int8_dgrad(dy.to(DEV), offd, packed, E, N, K, h1=h1.to(DEV), activation=act, save_dh1=False,
                                     dx=dx0.clone())
        assert none is None and torch.equal(dx2.view(torch.int16), dx.view(torch.int16))
    got = _f64(dx)
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        v = (g32[lo:hi] * ws[e].numpy()[None]).astype(np.float32).astype(np.float64)
        q, s = _quant(v)
        with np.errstate(invalid="ignore", divide="ignore"):
            t = np.nan_to_num(v * 127 / np.max(np.abs(v), axis=1, keepdims=True)) if hi > lo else v
        tie = (np.abs(t - np.floor(t) - 0.5) <= 127 * 4 * 2.0 ** -24).astype(np.float64)
        w = wq[e].double().numpy()
        _close(got[lo:hi], (q @ w) * s[:, None], extra=np.nan_to_num(s)[:, None] * (tie @ np.abs(w)))
    assert np.all(got[:lead] == 3) and np.all(got[M - tail:] == 3)


def test_wide_rows_are_computed_twice():
    """Widths past what a wavefront keeps in registers."""
    gg = _gg()
    for act, K, N in ((None, 8712, 40), ("swiglu", 4360, 40), (None, 40, 4360), ("swiglu", 40, 8720)):
        log(f"[int8] wide K={K} N={N} {act}")
        off = _offsets([2, 3])
        wq, ws = _weights(2, N, K, 3)
        offd = torch.from_numpy(off).to(DEV)
        if K > N:
            x = _rows(5, K if act is None else 2 * K, 1)
            y, a = gg.gg_int8_forward(x.to(DEV), offd, gg.gg_int8_pack(wq.to(DEV), ws.to(DEV)), 2, N, K, activation=act,
                                      save_a=act is not None)
            v = _f64(x if act is None else a)
            _close(_f64(y), _reference_forward(v, _quant(v), wq.double().numpy(), ws.double().numpy(), off))
        else:
            dy = _rows(5, N if act is None else N // 2, 1)
            h1 = None if act is None else _rows(5, N, 2).to(DEV)
            dx, dh1 = gg.gg_int8_dgrad(dy.to(DEV), offd, gg.gg_int8_pack_transposed(wq.to(DEV), ws.to(DEV)), 2, N, K, h1=h1,
                                       activation=act)
            g = (dy if act is None else dh1.cpu()).float().numpy()
            for e, (lo, hi) in enumerate(((0, 2), (2, 5))):
                v = (g[lo:hi] * ws[e].numpy()[None]).astype(np.float64)
                q, s = _quant(v)
                t = v * 127 / np.max(np.abs(v), axis=1, keepdims=True)
                tie = (np.abs(t - np.floor(t) - 0.5) <= 127 * 4 * 2.0 ** -24).astype(np.float64)
                w = wq[e].double().numpy()
                _close(_f64(dx)[lo:hi], (q @ w) * s[:, None], extra=s[:, None] * (tie @ np.abs(w)))


def test_rows_do_not_depend_on_the_batch():
    """A row's result is the same whether its expert owns 1 row or 700 (bit for bit)."""
    gg = _gg()
    K, N = 640, 776
    x = _rows(700, K, 21).to(DEV)
    wq, ws = _weights(1, N, K, 22)
    packed = gg.gg_int8_pack(wq.to(DEV), ws.to(DEV))
    whole, _ = gg.gg_int8_forward(x, torch.tensor([0, 700], device=DEV), packed, 1, N, K)
    for lo, hi in ((0, 1), (5, 37), (100, 195), (256, 612)):
        part, _ = gg.gg_int8_forward(x[lo:hi].contiguous(), torch.tensor([0, hi - lo], device=DEV), packed, 1, N, K)
        assert bitwise_equal(part, whole[lo:hi])


def test_other_stream_and_repeat():
    gg = _gg()
    off = torch.tensor([0, 130, 130, 171], device=DEV)
    x = _rows(171, 264, 31).to(DEV)
    wq, ws = _weights(3, 296, 264, 32)
    packed = gg.gg_int8_pack(wq.to(DEV), ws.to(DEV))
    first, _ = gg.gg_int8_forward(x, off, packed, 3, 296, 264)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    second, _ = gg.gg_int8_forward(x, off, packed, 3, 296, 264, stream=st)
    st.synchronize()
    assert bitwise_equal(first, second)


def test_binding_refuses():
    gg = _gg()
    wq, ws = (t.to(DEV) for t in _weights(2, 48, 64, 1))
    packed = gg.gg_int8_pack(wq, ws)
    x, off = _rows(4, 64, 1).to(DEV), torch.tensor([0, 2, 4], device=DEV)
    bad = [
        lambda: gg.gg_int8_forward(x.float(), off, packed, 2, 48, 64),
        lambda: gg.gg_int8_forward(x.cpu(), off, packed, 2, 48, 64),
        lambda: gg.gg_int8_forward(x[:, ::2], off, packed, 2, 48, 32),
        lambda: gg.gg_int8_forward(x, off.int(), packed, 2, 48, 64),
        lambda: gg.gg_int8_forward(x, off, packed[:100], 2, 48, 64),
        lambda: gg.gg_int8_forward(x, off, packed, 2, 48, 64, activation="relu"),
        lambda: gg.gg_int8_forward(x, off, packed, 2, 48, 64, activation="swiglu"),    # x is not [M, 2K]
        lambda: gg.gg_int8_forward(x, off, packed, 2, 48, 64, save_a=True),
        lambda: gg.gg_int8_forward(x, off, packed, 2, 48, 64, y=torch.empty(4, 40, dtype=torch.bfloat16, device=DEV)),
        lambda: gg.gg_int8_forward(x, off, packed, 2, 48, 64, workspace=torch.empty(8, device=DEV)),
        lambda: gg.gg_int8_dgrad(x, off, packed, 2, 64, 48, activation="swiglu"),       # no h1
        lambda: gg.gg_int8_dgrad(x, off, packed, 2, 64, 48, h1=x),
        lambda: gg.gg_int8_pack(wq.float(), ws),
        lambda: gg.gg_int8_pack(wq, ws[:, :40].contiguous()),
        lambda: gg.gg_int8_pack(wq[:, :, :60].contiguous(), ws),                        # K not a multiple of 8
        lambda: gg.gg_int8_quantize_rows(x[0]),
        lambda: gg.gg_int8_quantize_rows(x, q=torch.empty(4, 60, dtype=torch.int8, device=DEV)),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was accepted")

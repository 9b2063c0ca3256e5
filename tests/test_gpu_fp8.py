"""GPU: the block-scaled 8-bit floating-point products (gg_fp8_*) against
their definition in 64 bits on the CPU.

Tolerances: quantization is exact, so products by an identity matrix are
compared bit for bit; other products are within fp8_reference.bound (the matrix
instruction's sums, one rounding to bf16).  A and dH1: the sigmoid's exponential and
reciprocal are within 2^-19 for |gate| <= 16, a derivative sums two such
terms; then bf16 (2^-8)."""
import numpy as np
import pytest
import torch

import fp8_reference as ref
from gpu_harness import bitwise_equal, log

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _gg():
    import moe_expert_grouped_ragged_amd as gg
    return gg


def _f64(t):
    return t.detach().cpu().double().numpy()


def _bytes(s):
    return s.cpu().view(torch.uint8).numpy()


def _rows(M, K, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(M, K, generator=g) * torch.exp(0.7 * torch.randn(M, 1, generator=g)) * torch.exp(torch.randn(K, generator=g))
    return x.to(torch.bfloat16)


def _weights(E, N, K, halves, seed):
    """(q, s, the matrices they stand for) of random weights, by the definition."""
    g = torch.Generator().manual_seed(seed)
    w = (torch.randn(E, N, K, generator=g) * torch.exp(torch.randn(E, N, 1, generator=g)) * 0.02).to(torch.bfloat16)
    both = [ref.quant_weights(m, halves) for m in w.double().numpy()]
    q = torch.from_numpy(np.stack([b[0] for b in both])).float().to(torch.float8_e4m3fn)
    s = torch.from_numpy(np.stack([b[1] for b in both]))
    return w, q.to(DEV), s.view(torch.float8_e8m0fnu).to(DEV), [ref.dequant(*b, halves) for b in both]


def _offsets(counts, lead=0):
    return np.concatenate([[lead], lead + np.cumsum(counts)]).astype(np.int64)


def _experts(off):
    return [(e, int(a), int(b)) for e, (a, b) in enumerate(zip(off, off[1:])) if b > a]


def _off(off):
    return torch.from_numpy(off).to(DEV)


def _within(got, want, bound, what):
    assert np.array_equal(np.isnan(got), np.isnan(want)), what
    m = ~np.isnan(want)
    err = np.abs(got - want)[m]
    worst = float(np.max(err / bound[m])) if err.size else 0.0
    log(f"[fp8] {what}: worst {worst:.3f} of the bound")
    assert worst <= 1.0, what


COUNTS = [0, 1, 33, 2, 130, 0, 64, 300, 7]


@pytest.mark.parametrize("N,K,halves", [(8, 8, 1), (136, 264, 1), (128, 128, 1), (272, 520, 2), (304, 136, 2), (16, 136, 2)])
def test_weight_quantization(N, K, halves):
    gg = _gg()
    w, q, s, _ = _weights(3, N, K, halves, 5)
    w[1, :, :] *= 1e-3
    w[2, 0, :8] = torch.tensor([448, 449, 1.75, 2.0 ** -130, 0, -448, 3e38, -1e-30]).to(torch.bfloat16)
    w[0, -1, 0] = float("nan")
    gq, gs = gg.gg_fp8_quantize_weights(w.to(DEV), halves=halves)
    assert tuple(gs.shape) == gg.fp8_scale_shape(3, N, K, halves) and gs.numel() == gg.lib.gg_fp8_scale_bytes(3, N, K, halves)
    for e in range(3):
        m = w[e].double().numpy()
        if e == 0:
            m = m.copy()
            m[-1, 0] = 0
        want, ws = ref.quant_weights(m, halves)
        got, gb = gq[e].cpu().float().double().numpy(), _bytes(gs[e])
        if e == 0:     # the block with the NaN is all NaN, with scale one
            r, c = ref.spans(N, halves)[-1], ref.spans(K)[0]
            assert np.isnan(got[r, c]).all() and gb[-1, 0] == 127
            want[r, c], ws[-1, 0] = np.nan, 127
        assert np.array_equal(got, want, equal_nan=True) and np.array_equal(gb, ws), e


SPECIAL = [0.0, -0.0, 448.0, 449.0, 1.75, 1.7578125, 2.0 ** -133, -2.0 ** -126, 3.3e38, 2.0 ** -6, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10]


@pytest.mark.parametrize("K", [8, 128, 136, 520])
def test_rows_are_quantized_as_defined(K):
    """Products by an identity matrix with scales one are what the quantized rows stand for, bit for bit."""
    gg = _gg()
    M = 301
    x = _rows(M, K, 3)
    g = torch.Generator().manual_seed(9)
    for i, v in enumerate(SPECIAL):
        x[2 * i, :] = v
        x[2 * i + 1, : K // 2] = v
    # every significand against every other: the borders of the scale, ties and subnormal results
    x[100:200] = (torch.randint(-255, 256, (100, K), generator=g).float() * torch.exp2(torch.randint(-12, 4, (100, K), generator=g).float())).to(torch.bfloat16)
    x[210, 0], x[211, K - 1], x[212, 3] = float("nan"), float("inf"), float("-inf")
    x[213] = 0
    eye = torch.eye(K).to(torch.float8_e4m3fn).view(1, K, K).to(DEV)
    s = torch.full(gg.fp8_scale_shape(1, K, K), 127, dtype=torch.uint8, device=DEV).view(torch.float8_e8m0fnu)
    lo, hi = 3, M - 2
    off = _off(np.array([lo, hi], np.int64))
    want = ref.quant(x.double().numpy())
    # 1.9375 * 2^127 (the bf16 value of 3.3e38) rounds to 256 * 2^120 = 2^128, which fp32 and bf16 hold as infinity
    want = np.where(np.abs(want) >= 2.0 ** 128, np.copysign(np.inf, want), want)
    for call in (lambda y: gg.gg_fp8_forward(x.to(DEV), off, gg.gg_fp8_pack(eye, s), 1, K, K, y=y),
                 lambda y: gg.gg_fp8_dgrad(x.to(DEV), off, gg.gg_fp8_pack_transposed(eye, s), 1, K, K, dx=y)):
        y = torch.full((M, K), 7.0, dtype=torch.bfloat16, device=DEV)
        call(y)
        got = _f64(y)
        assert np.all(got[:lo] == 7) and np.all(got[hi:] == 7)
        for r in range(lo, hi):
            if np.isnan(want[r]).any():
                assert np.isnan(got[r]).all(), r       # a NaN times zero is in every sum
                continue
            # the instruction may flush what lies below fp32's normal numbers
            assert np.array_equal(np.where(np.abs(want[r]) < 2.0 ** -126, 0, want[r]),
                                  np.where(np.abs(got[r]) < 2.0 ** -126, 0, got[r])), r


@pytest.mark.parametrize("N,K,halves", [(8, 8, 1), (40, 264, 1), (256, 128, 1), (392, 520, 1), (304, 136, 2), (528, 1032, 2), (16, 2056, 2)])
def test_forward(N, K, halves):
    gg = _gg()
    off = _offsets(COUNTS, lead=5)
    M = int(off[-1]) + 6
    x = _rows(M, K, N + K)
    _, q, s, w = _weights(len(COUNTS), N, K, halves, 11)
    y = torch.full((M, N), 7.0, dtype=torch.bfloat16, device=DEV)
    out, a = gg.gg_fp8_forward(x.to(DEV), _off(off), gg.gg_fp8_pack(q, s, halves=halves), len(COUNTS), N, K, halves=halves, y=y)
    assert out is y and a is None
    got = _f64(y)
    assert np.all(got[:5] == 7) and np.all(got[-6:] == 7)
    for e, lo, hi in _experts(off):
        want, err = ref.product(ref.quant(x[lo:hi].double().numpy()), w[e])
        _within(got[lo:hi], want, ref.bound(want, err), f"forward {N}x{K} expert {e}")


@pytest.mark.parametrize("N,K,halves", [(8, 8, 1), (264, 40, 1), (128, 256, 1), (304, 136, 2), (1040, 392, 2)])
def test_dgrad(N, K, halves):
    gg = _gg()
    off = _offsets(COUNTS, lead=3)
    M = int(off[-1]) + 1
    dy = _rows(M, N, N + K)
    _, q, s, w = _weights(len(COUNTS), N, K, halves, 12)
    dx = torch.full((M, K), 7.0, dtype=torch.bfloat16, device=DEV)
    gg.gg_fp8_dgrad(dy.to(DEV), _off(off), gg.gg_fp8_pack_transposed(q, s, halves=halves), len(COUNTS), N, K, halves=halves, dx=dx)
    got = _f64(dx)
    assert np.all(got[:3] == 7) and np.all(got[-1:] == 7)
    for e, lo, hi in _experts(off):
        want, err = ref.product(ref.quant(dy[lo:hi].double().numpy(), halves), w[e].T)
        _within(got[lo:hi], want, ref.bound(want, err), f"dgrad {N}x{K} expert {e}")


@pytest.mark.parametrize("act", ["swiglu", "qgeglu"])
@pytest.mark.parametrize("N,F", [(40, 136), (264, 520), (128, 8)])
def test_forward_with_the_activation_in_front(N, F, act):
    gg = _gg()
    off = _offsets(COUNTS, lead=2)
    M, E, k = int(off[-1]) + 3, len(COUNTS), ref.SLOPE[act]
    h1 = _rows(M, 2 * F, 4).clamp(-16, 16)
    _, q, s, w = _weights(E, N, F, 1, 13)
    packed = gg.gg_fp8_pack(q, s)
    a_out = torch.full((M, F), 7.0, dtype=torch.bfloat16, device=DEV)
    y, a = gg.gg_fp8_forward(h1.to(DEV), _off(off), packed, E, N, F, activation=act, a_out=a_out)
    y2, none = gg.gg_fp8_forward(h1.to(DEV), _off(off), packed, E, N, F, activation=act)
    live = slice(int(off[0]), int(off[-1]))
    assert none is None and bitwise_equal(y[live], y2[live])
    ga, gy = _f64(a), _f64(y)
    assert np.all(ga[:2] == 7) and np.all(ga[-3:] == 7)
    want = ref.act(h1.double().numpy(), k)
    _within(ga[live], want[live], (2.0 ** -8 + 2.0 ** -18) * np.abs(want[live]) + 1e-37, "A")
    for e, lo, hi in _experts(off):
        want, err = ref.product(ref.quant(ga[lo:hi]), w[e])          # of the A that was returned
        _within(gy[lo:hi], want, ref.bound(want, err), f"act forward expert {e}")


@pytest.mark.parametrize("act", ["swiglu", "qgeglu"])
@pytest.mark.parametrize("F,K", [(136, 40), (520, 264), (8, 128)])
def test_dgrad_with_the_derivative_in_front(F, K, act):
    gg = _gg()
    off = _offsets(COUNTS, lead=2)
    M, E, k = int(off[-1]) + 3, len(COUNTS), ref.SLOPE[act]
    h1, da = _rows(M, 2 * F, 5).clamp(-16, 16), _rows(M, F, 6)
    _, q, s, w = _weights(E, 2 * F, K, 2, 14)
    packed = gg.gg_fp8_pack_transposed(q, s, halves=2)
    args = (da.to(DEV), _off(off), packed, E, 2 * F, K)
    dx, dh = gg.gg_fp8_dgrad(*args, halves=2, h1=h1.to(DEV), activation=act)
    dx2, none = gg.gg_fp8_dgrad(*args, halves=2, h1=h1.to(DEV), activation=act, save_dh1=False)
    live = slice(int(off[0]), int(off[-1]))
    assert none is None and bitwise_equal(dx[live], dx2[live])
    gd, gx = _f64(dh), _f64(dx)
    h, d = h1.double().numpy(), da.double().numpy()
    want = ref.act_grad(h, d, k)
    g, u = np.split(h, 2, axis=1)
    sg = 1 / (1 + np.exp(-k * g))
    terms = np.concatenate([np.abs(d * u) * sg * (1 + np.abs(k * g) * (1 - sg)), np.abs(d * g) * sg], axis=1)
    _within(gd[live], want[live], 2.0 ** -8 * np.abs(want[live]) + 2.0 ** -17 * terms[live] + 1e-37, "dH1")
    for e, lo, hi in _experts(off):
        want, err = ref.product(ref.quant(gd[lo:hi], 2), w[e].T)
        _within(gx[lo:hi], want, ref.bound(want, err), f"act dgrad expert {e}")


BLOCKS = [(COUNTS, 136, 152, "swiglu"), (COUNTS, 264, 128, "qgeglu"), ([1] * 8, 512, 384, "swiglu"), ([40, 0, 3], 1032, 8, "qgeglu"),
          ([700, 0, 256, 90, 300], 256, 264, "swiglu")]


def _block_weights(gg, E, H, F, seed):
    g = torch.Generator().manual_seed(seed)
    w1 = (torch.randn(E, 2 * F, H, generator=g) / H ** 0.5).to(torch.bfloat16).to(DEV)
    w2 = (torch.randn(E, H, F, generator=g) / F ** 0.5).to(torch.bfloat16).to(DEV)
    return gg.fp8_experts(w1, w2)


@pytest.mark.parametrize("counts,H,F,act", BLOCKS)
def test_gated_block_is_its_single_calls(counts, H, F, act):
    """The gated block, forward and backward, gives the bits of the single calls in a row, with and without H1
    saved, and leaves the rows outside alone."""
    gg = _gg()
    off = _offsets(counts, lead=3)
    M, E = int(off[-1]) + 4, len(counts)
    live, o = slice(int(off[0]), int(off[-1])), _off(off)
    w = _block_weights(gg, E, H, F, 21)
    x, dy = _rows(M, H, 22).to(DEV), _rows(M, H, 23).to(DEV)
    h1, _ = gg.gg_fp8_forward(x, o, w.fc1, E, 2 * F, H, halves=2)
    y, _ = gg.gg_fp8_forward(h1, o, w.fc2, E, H, F, activation=act)
    da, _ = gg.gg_fp8_dgrad(dy, o, w.fc2_t, E, H, F)
    dx, _ = gg.gg_fp8_dgrad(da, o, w.fc1_t, E, 2 * F, H, halves=2, h1=h1, activation=act)

    def seven(width):
        return torch.full((M, width), 7.0, dtype=torch.bfloat16, device=DEV)

    by, bh, by2, bx = seven(H), seven(2 * F), seven(H), seven(H)
    gg.gg_fp8_glu_forward(x, o, w.fc1, w.fc2, E, H, F, activation=act, h1_out=bh, y=by)
    _, none = gg.gg_fp8_glu_forward(x, o, w.fc1, w.fc2, E, H, F, activation=act, save_h1=False, y=by2)
    gg.gg_fp8_glu_dgrad(dy, bh, o, w.fc1_t, w.fc2_t, E, H, F, activation=act, dx=bx)
    assert none is None
    for name, got, want in (("h1", bh, h1), ("y", by, y), ("y without h1", by2, y), ("dx", bx, dx)):
        assert bitwise_equal(got[live], want[live]), name
        outside = torch.cat([got[:3], got[-4:]])
        assert bool((outside == 7).all()), name


@pytest.mark.parametrize("K,N", [(264, 392), (2048, 256)])
def test_a_rows_bits_do_not_depend_on_the_batch(K, N):
    """The same rows alone, in small and in large experts, and among many experts."""
    gg = _gg()
    x = _rows(700, K, 31).to(DEV)
    _, q, s, _ = _weights(1, N, K, 1, 32)
    want, _ = gg.gg_fp8_forward(x, _off(np.array([0, 700], np.int64)), gg.gg_fp8_pack(q, s), 1, N, K)
    for counts in ([1] * 700, [96, 97, 64, 65, 32, 33, 128, 129, 56], [256, 300, 144]):
        E = len(counts)
        qs, ss = (t.view(torch.uint8).expand(E, *t.shape[1:]).contiguous() for t in (q, s))
        packed = gg.gg_fp8_pack(qs.view(torch.float8_e4m3fn), ss.view(torch.float8_e8m0fnu))
        got, _ = gg.gg_fp8_forward(x, _off(_offsets(counts)), packed, E, N, K)
        assert bitwise_equal(got, want), counts


def test_not_finite_values_stay_in_their_rows():
    gg = _gg()
    E, H, F, M = 2, 264, 136, 300
    w = _block_weights(gg, E, H, F, 41)
    o = _off(np.array([0, 140, M], np.int64))
    x = _rows(M, H, 42).to(DEV)
    y, h1 = gg.gg_fp8_glu_forward(x, o, w.fc1, w.fc2, E, H, F)
    bad = x.clone()
    bad[5, 0], bad[150, H - 1], bad[299, 130] = float("nan"), float("inf"), float("-inf")
    by, bh = gg.gg_fp8_glu_forward(bad, o, w.fc1, w.fc2, E, H, F)
    dx, bx = (gg.gg_fp8_glu_dgrad(t, h1, o, w.fc1_t, w.fc2_t, E, H, F) for t in (x, bad))
    rows = torch.tensor([5, 150, 299], device=DEV)
    keep = torch.ones(M, dtype=torch.bool, device=DEV)
    keep[rows] = False
    for got, want in ((by, y), (bh, h1), (bx, dx)):
        assert bool(torch.isnan(got[rows]).all()) and bitwise_equal(got[keep], want[keep])


def test_no_rows():
    gg = _gg()
    w = _block_weights(gg, 3, 64, 40, 51)
    none = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV)
    o = torch.zeros(4, dtype=torch.int64, device=DEV)
    y, h1 = gg.gg_fp8_glu_forward(none, o, w.fc1, w.fc2, 3, 64, 40)
    assert y.shape == (0, 64) and h1.shape == (0, 80)
    assert gg.gg_fp8_glu_dgrad(none, h1, o, w.fc1_t, w.fc2_t, 3, 64, 40).shape == (0, 64)
    # rows, but no expert owns one (also where their common offset is odd)
    x = _rows(9, 64, 52).to(DEV)
    for at in (0, 3, 9):
        y = torch.full((9, 64), 7.0, dtype=torch.bfloat16, device=DEV)
        gg.gg_fp8_glu_forward(x, torch.full((4,), at, dtype=torch.int64, device=DEV), w.fc1, w.fc2, 3, 64, 40, y=y)
        assert bool((y == 7).all())

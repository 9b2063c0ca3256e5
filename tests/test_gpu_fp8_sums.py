"""GPU: how the 8-bit floating-point products add up (fp32 sums, the scaled instruction's), value by value:
planted values, H1 and dA as they round to bf16, and the gated block's outputs, each held to the 64-bit
definition by the intervals of fp8_sums_reference."""
import numpy as np
import pytest
import torch

import fp8_reference as ref
import fp8_sums_reference as sums
from gpu_harness import bitwise_equal, log

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
ZIPF = [150, 0, 71, 33, 17, 9, 0, 5, 1]


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _gg():
    import moe_expert_grouped_ragged_amd as gg
    return gg


def _f64(t):
    return t.detach().cpu().double().numpy()


def _off(counts, lead=0):
    return np.concatenate([[lead], lead + np.cumsum(counts)]).astype(np.int64)


def _dev(off):
    return torch.from_numpy(off).to(DEV)


def _rows(M, K, seed):
    """Rows and channels of uneven size."""
    g = torch.Generator().manual_seed(seed)
    gain = torch.exp(0.5 * torch.randn(M, 1, generator=g)) * torch.exp(0.5 * torch.randn(K, generator=g))
    return (torch.randn(M, K, generator=g) * gain).to(torch.bfloat16)


def _weights(E, N, K, halves, seed):
    """(q, s, the matrices they stand for)."""
    g = torch.Generator().manual_seed(seed)
    w = (torch.randn(E, N, K, generator=g) * 0.02).to(torch.bfloat16).double().numpy()
    both = [ref.quant_weights(m, halves) for m in w]
    q = torch.from_numpy(np.stack([b[0] for b in both])).float().to(torch.float8_e4m3fn)
    s = torch.from_numpy(np.stack([b[1] for b in both]))
    return q.to(DEV), s.view(torch.float8_e8m0fnu).to(DEV), [ref.dequant(*b, halves) for b in both]


def _within(got, lo, hi, what):
    out = int(np.sum((got < lo) | (got > hi)))
    log(f"[fp8 sums] {what}: {out} of {got.size} outside, {np.mean(lo == hi):.4f} known exactly")
    assert out == 0, what


def _ends(got, dev, err):
    """The values that bf16(got +- (dev + err)) may be."""
    return sums.bf16(got - dev - err), sums.bf16(got + dev + err)


@pytest.mark.parametrize("M", [1, 40, 300])
@pytest.mark.parametrize("K", [8, 264, 2048])
def test_planted_values_cancel(M, K):
    """(256, 256, 2) times (256, -256, 2) is 4, wherever the three lie among the summed columns, for small batches and
    tiles, in H1 and dA and wherever fp32 sums are asked for."""
    gg = _gg()
    N = 144
    places = [(0, 1, 2), (7, 5, 0), (K - 1, K - 8, K - 4), (K - 8, K - 7, K - 1)]
    x = torch.zeros(M, K)
    for r in range(M):
        a, b, c = places[r % len(places)]
        x[r, a], x[r, b], x[r, c] = 256.0, 256.0, 2.0
    o = _dev(np.array([0, M], np.int64))
    one = gg.fp8_scale_shape
    for r, (a, b, c) in enumerate(places[:min(M, len(places))]):
        w = torch.zeros(1, N, K)
        w[:, :, a], w[:, :, b], w[:, :, c] = 256.0, -256.0, 2.0
        want = x @ w[0, 0]                     # 4 in this place's rows, whole numbers in all
        q = w.to(torch.float8_e4m3fn).to(DEV)
        xd = x.to(torch.bfloat16).to(DEV)

        def scale(*shape, halves=1):
            return torch.full(one(*shape, halves), 127, dtype=torch.uint8, device=DEV).view(torch.float8_e8m0fnu)

        qt = w.transpose(1, 2).contiguous().to(torch.float8_e4m3fn).to(DEV)
        fwd1, fwd2 = gg.gg_fp8_pack(q, scale(1, N, K)), gg.gg_fp8_pack(q, scale(1, N, K, halves=2), halves=2)
        back = gg.gg_fp8_pack_transposed(qt, scale(1, K, N))
        for got in (gg.gg_fp8_forward(xd, o, fwd2, 1, N, K, halves=2)[0],
                    gg.gg_fp8_forward(xd, o, fwd1, 1, N, K, sums="fp32")[0],
                    gg.gg_fp8_dgrad(xd, o, back, 1, K, N)[0],
                    gg.gg_fp8_dgrad(xd, o, back, 1, K, N, sums="fp32")[0]):
            assert torch.equal(got.cpu(), want[:, None].to(torch.bfloat16).expand(M, N)), (r, a, b, c)


@pytest.mark.parametrize("how", ["fp32", "scaled"])
@pytest.mark.parametrize("counts,N,K,halves", [(ZIPF, 136, 264, 1), (ZIPF, 304, 136, 2), ([1] * 8 + [0, 3], 272, 2056, 2), (ZIPF, 40, 520, 1)])
def test_both_sums_of_both_directions(how, counts, N, K, halves):
    gg = _gg()
    off = _off(counts, 3)
    M, E = int(off[-1]) + 2, len(counts)
    o = _dev(off)
    q, s, w = _weights(E, N, K, halves, 31)
    x, dy = _rows(M, K, 32), _rows(M, N, 33)
    y, dx = (torch.full((M, n), 7.0, dtype=torch.bfloat16, device=DEV) for n in (N, K))
    gg.gg_fp8_forward(x.to(DEV), o, gg.gg_fp8_pack(q, s, halves=halves), E, N, K, halves=halves, y=y, sums=how)
    gg.gg_fp8_dgrad(dy.to(DEV), o, gg.gg_fp8_pack_transposed(q, s, halves=halves), E, N, K, halves=halves, dx=dx, sums=how)
    for got, rows, h, t in ((y, x, 1, False), (dx, dy, halves, True)):
        got = _f64(got)
        assert np.all(got[:3] == 7) and np.all(got[-2:] == 7)
        for e in range(E):
            lo, hi = int(off[e]), int(off[e + 1])
            if lo < hi:
                v, m = ref.quant(rows[lo:hi].double().numpy(), h), w[e].T if t else w[e]
                want, err = sums.fp32_sums(v, m) if how == "fp32" else ref.product(v, m)
                _within(got[lo:hi], *_ends(want, 0, err), f"{how} {'dx' if t else 'y'} {N}x{K} expert {e}")


@pytest.mark.parametrize("act", ["swiglu", "qgeglu"])
@pytest.mark.parametrize("how", [None, "fp32"])
def test_a_zipf_batch_through_the_block(how, act):
    """Forward: H1 to the definition; y to the definition on that H1, where A and its e4m3 values may be any that the
    activation's error (2^-18 of A) leaves open.  Backward: dA by the single product to the definition; dx to the
    definition, where dA may be any that its sums leave open, dH1 any within 2^-17 of its terms of those, and its e4m3
    values any of those.  Then the error of y and dx over all, most of which is the last rounding."""
    gg = _gg()
    H, F, k = 2048, 768, ref.SLOPE[act]
    off = _off(ZIPF, 2)
    M, E = int(off[-1]) + 1, len(ZIPF)
    o = _dev(off)
    q1, s1, w1 = _weights(E, 2 * F, H, 2, 41)
    q2, s2, w2 = _weights(E, H, F, 1, 42)
    x, dy = _rows(M, H, 43), _rows(M, H, 44)
    fc2_t = gg.gg_fp8_pack_transposed(q2, s2)
    y, h1 = gg.gg_fp8_glu_forward(x.to(DEV), o, gg.gg_fp8_pack(q1, s1, halves=2), gg.gg_fp8_pack(q2, s2), E, H, F, act, sums=how)
    dx = gg.gg_fp8_glu_dgrad(dy.to(DEV), h1, o, gg.gg_fp8_pack_transposed(q1, s1, halves=2), fc2_t, E, H, F, act, sums=how)
    da, _ = gg.gg_fp8_dgrad(dy.to(DEV), o, fc2_t, E, H, F, sums=how)
    gy, gh, gx, ga = _f64(y), _f64(h1), _f64(dx), _f64(da)
    last = sums.fp32_sums if how == "fp32" else ref.product
    square = {"y": [0.0, 0.0], "dx": [0.0, 0.0]}

    def count(name, got, want):
        square[name][0] += float(np.sum((got - want) ** 2))
        square[name][1] += float(np.sum(want ** 2))

    for e in range(E):
        r = slice(int(off[e]), int(off[e + 1]))
        if r.start == r.stop:
            continue
        want, err = sums.fp32_sums(ref.quant(x[r].double().numpy()), w1[e])
        _within(gh[r], *_ends(want, 0, err), f"H1, expert {e}")
        a = ref.act(gh[r], k)
        v, dev = sums.quant_interval(sums.bf16(a - 2.0 ** -18 * np.abs(a)), sums.bf16(a + 2.0 ** -18 * np.abs(a)))
        want, err = last(v, w2[e])
        err = err + 2.0 ** -10 * (dev @ np.abs(w2[e]).T)      # the sums of other values have other errors, within their size
        _within(gy[r], *_ends(want, dev @ np.abs(w2[e]).T, err), f"y, expert {e}")
        count("y", gy[r], ref.quant(sums.bf16(a)) @ w2[e].T)

        want, err = sums.fp32_sums(ref.quant(dy[r].double().numpy()), w2[e].T)
        lo, hi = _ends(want, 0, err)
        _within(ga[r], lo, hi, f"dA, expert {e}")
        g, u = np.split(gh[r], 2, axis=1)
        sg = 1 / (1 + np.exp(-k * g))
        terms = np.concatenate([np.abs(u) * sg * (1 + np.abs(k * g) * (1 - sg)), np.abs(g) * sg], axis=1)
        slack = 2.0 ** -17 * terms * np.tile(np.maximum(np.abs(lo), np.abs(hi)), 2)
        ends = [ref.act_grad(gh[r], t, k) for t in (lo, hi)]           # linear in dA
        v, dev = sums.quant_interval(sums.bf16(np.minimum(*ends) - slack), sums.bf16(np.maximum(*ends) + slack), 2)
        want, err = last(v, w1[e].T)
        err = err + 2.0 ** -10 * (dev @ np.abs(w1[e]))
        _within(gx[r], *_ends(want, dev @ np.abs(w1[e]), err), f"dx, expert {e}")
        count("dx", gx[r], ref.quant(sums.bf16(ref.act_grad(gh[r], ga[r], k)), 2) @ w1[e])
    for name, (num, den) in square.items():
        rel = (num / den) ** 0.5
        log(f"[fp8 sums] {name}: {rel:.5f} of the norm")
        # rounding to bf16 is off by up to 2^-8 of the value's power of two, evenly: 2^-8 / sqrt(3) in the mean square of
        # values that are at least that power
        assert rel <= 2.0 ** -8 / 3 ** 0.5, (name, rel)


@pytest.mark.parametrize("how", ["fp32", "scaled"])
@pytest.mark.parametrize("counts,H,F", [([40, 0, 3, 1], 264, 136), ([1] * 8, 512, 384), ([700, 0, 256, 90, 300], 256, 264),
                                        ([1500, 33, 1900], 264, 2048), ([1024, 0, 257, 1, 352, 609, 96, 33, 511], 136, 2040)])
def test_the_block_is_its_single_calls_of_the_same_sums(how, counts, H, F):
    gg = _gg()
    E, act = len(counts), "swiglu"
    off = _off(counts, 3)
    M, o = int(off[-1]) + 2, _dev(off)
    live = slice(3, int(off[-1]))
    g = torch.Generator(device=DEV).manual_seed(51)
    n = lambda *s: torch.randn(s, generator=g, device=DEV)      # noqa: E731
    w = gg.fp8_experts((n(E, 2 * F, H) / H ** 0.5).to(torch.bfloat16), (n(E, H, F) / F ** 0.5).to(torch.bfloat16))
    x, dy = n(M, H).to(torch.bfloat16), n(M, H).to(torch.bfloat16)
    h1, _ = gg.gg_fp8_forward(x, o, w.fc1, E, 2 * F, H, halves=2, sums=how)
    y, _ = gg.gg_fp8_forward(h1, o, w.fc2, E, H, F, activation=act, sums=how)
    da, _ = gg.gg_fp8_dgrad(dy, o, w.fc2_t, E, H, F, sums=how)
    dx, _ = gg.gg_fp8_dgrad(da, o, w.fc1_t, E, 2 * F, H, halves=2, h1=h1, activation=act, sums=how)
    by, bh, bx = (torch.full((M, width), 7.0, dtype=torch.bfloat16, device=DEV) for width in (H, 2 * F, H))
    gg.gg_fp8_glu_forward(x, o, w.fc1, w.fc2, E, H, F, activation=act, h1_out=bh, y=by, sums=how)
    gg.gg_fp8_glu_dgrad(dy, bh, o, w.fc1_t, w.fc2_t, E, H, F, activation=act, dx=bx, sums=how)
    for name, got, want in (("h1", bh, h1), ("y", by, y), ("dx", bx, dx)):
        assert bitwise_equal(got[live], want[live]), name
        assert bool((got[:3] == 7).all()) and bool((got[-2:] == 7).all()), name


@pytest.mark.parametrize("how", ["fp32", "scaled"])
@pytest.mark.parametrize("K,N", [(264, 392), (2048, 256), (4104, 136)])
def test_a_rows_bits_do_not_depend_on_the_batch(how, K, N):
    """Rows alone, streamed, and in tiles of each size (256 x 256 of 3400 rows)."""
    gg = _gg()
    x = _rows(3400, K, 61).to(DEV)
    q, s, _ = _weights(1, N, K, 1, 62)
    want, _ = gg.gg_fp8_forward(x, _dev(np.array([0, 3400], np.int64)), gg.gg_fp8_pack(q, s), 1, N, K, sums=how)
    for counts in ([1] * 700 + [2700], [96, 97, 64, 65, 32, 33, 128, 129, 2756], [256, 300, 144, 2700]):
        E = len(counts)
        qs, ss = (t.view(torch.uint8).expand(E, *t.shape[1:]).contiguous() for t in (q, s))
        packed = gg.gg_fp8_pack(qs.view(torch.float8_e4m3fn), ss.view(torch.float8_e8m0fnu))
        got, _ = gg.gg_fp8_forward(x, _dev(_off(counts)), packed, E, N, K, sums=how)
        assert bitwise_equal(got, want), len(counts)
    small, _ = gg.gg_fp8_forward(x[:40].contiguous(), _dev(np.array([0, 40], np.int64)), gg.gg_fp8_pack(q, s), 1, N, K, sums=how)
    assert bitwise_equal(small, want[:40])


@pytest.mark.parametrize("how", ["fp32", "scaled"])
@pytest.mark.parametrize("M", [40, 301])
def test_scales_at_the_ends_of_their_range(how, M):
    """Rows and weights of the largest and smallest sizes through an identity matrix: what the quantized row stands for
    times the weights' scale (0 to 2^118 for fp32 sums), bit for bit where that is a normal number."""
    gg = _gg()
    K = 136
    eye = torch.eye(K).to(torch.float8_e4m3fn).view(1, K, K).to(DEV)
    o = _dev(np.array([0, M], np.int64))
    for c, rows in ((0, [2.0 ** 127, 1.99 * 2.0 ** 127, -3.0 * 2.0 ** 100]), (1, [2.0 ** 100, 3.3e38]), (126, [2.0 ** -100, 2.0 ** -126, 3.3e38]),
                    (127, [3.3e38, 2.0 ** -126, 2.0 ** -133, 0.0]), (200, [2.0 ** -126, 2.0 ** -80, 7 * 2.0 ** 50]), (245, [2.0 ** -126, 2.0 ** -120, 5.0])):
        x = torch.zeros(M, K, dtype=torch.bfloat16)
        for r in range(M):
            x[r] = rows[r % len(rows)]
            x[r, 1::3] = rows[r % len(rows)] / 4
        s = torch.full(gg.fp8_scale_shape(1, K, K), c, dtype=torch.uint8, device=DEV).view(torch.float8_e8m0fnu)
        want = ref.quant(x.double().numpy()) * 2.0 ** (c - 127)
        want = np.where(np.abs(want) >= 2.0 ** 128 * (1 - 2.0 ** -9), np.copysign(np.inf, want), want)
        for call in (lambda: gg.gg_fp8_forward(x.to(DEV), o, gg.gg_fp8_pack(eye, s), 1, K, K, sums=how)[0],
                     lambda: gg.gg_fp8_dgrad(x.to(DEV), o, gg.gg_fp8_pack_transposed(eye, s), 1, K, K, sums=how)[0]):
            got = _f64(call())
            ok = (got == want) | ((np.abs(got) < 2.0 ** -126) & (np.abs(want) < 2.0 ** -126))
            assert ok.all(), (c, got[~ok][:4], want[~ok][:4])


def test_unknown_sums_are_refused():
    gg = _gg()
    w = gg.fp8_experts(*(torch.ones(1, *s, dtype=torch.bfloat16, device=DEV) for s in ((16, 8), (8, 8))))
    x, o = torch.ones(4, 8, dtype=torch.bfloat16, device=DEV), _dev(np.array([0, 4], np.int64))
    for call in (lambda s: gg.gg_fp8_forward(x, o, w.fc1, 1, 16, 8, halves=2, sums=s), lambda s: gg.gg_fp8_dgrad(x, o, w.fc2_t, 1, 8, 8, sums=s),
                 lambda s: gg.gg_fp8_glu_forward(x, o, w.fc1, w.fc2, 1, 8, 8, sums=s),
                 lambda s: gg.gg_fp8_glu_dgrad(x, x.repeat(1, 2), o, w.fc1_t, w.fc2_t, 1, 8, 8, sums=s)):
        call("fp32")
        for bad in ("bf16", 1, ""):
            with pytest.raises(ValueError, match="sums"):
                call(bad)

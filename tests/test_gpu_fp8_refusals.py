"""GPU: what the binding of the block-scaled 8-bit products refuses (types, shapes,
strides, other layouts), and wrong offsets, which stay in bounds."""
import pytest
import torch

from gpu_harness import bitwise_equal, log

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
E, N, K = 2, 64, 64


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _normal(*shape):
    g = torch.Generator(device=DEV).manual_seed(len(shape) + sum(shape))
    return torch.randn(shape, generator=g, device=DEV).to(torch.bfloat16)


@pytest.fixture
def made():
    import moe_expert_grouped_ragged_amd as gg
    q, s = gg.gg_fp8_quantize_weights(_normal(E, N, K))
    return gg, q, s, _normal(5, K), torch.tensor([0, 2, 5], device=DEV)


def test_types_shapes_and_strides(made):
    gg, q, s, x, off = made
    p = gg.gg_fp8_pack(q, s)
    wide = _normal(5, 2 * K)
    for call in (
            lambda: gg.gg_fp8_quantize_weights(_normal(E, N, K).float()),
            lambda: gg.gg_fp8_quantize_weights(_normal(N, K)),
            lambda: gg.gg_fp8_quantize_weights(_normal(E, N, 60)),
            lambda: gg.gg_fp8_quantize_weights(_normal(E, 24, K), halves=2),
            lambda: gg.gg_fp8_quantize_weights(_normal(E, N, K), halves=3),
            lambda: gg.gg_fp8_pack(q.view(torch.uint8), s),
            lambda: gg.gg_fp8_pack(q, s.view(torch.uint8)),
            lambda: gg.gg_fp8_pack(q, s, halves=2),                       # other scales
            lambda: gg.gg_fp8_pack(q.transpose(1, 2), s),
            lambda: gg.gg_fp8_forward(x.float(), off, p, E, N, K),
            lambda: gg.gg_fp8_forward(wide[:, :K], off, p, E, N, K),      # a strided operand
            lambda: gg.gg_fp8_forward(wide, off, p, E, N, K),
            lambda: gg.gg_fp8_forward(x, off.int(), p, E, N, K),
            lambda: gg.gg_fp8_forward(x, off, p[:64], E, N, K),
            lambda: gg.gg_fp8_forward(x, off, p, E, N, K, save_a=True),
            lambda: gg.gg_fp8_forward(x, off, p, E, N, K, activation="relu"),
            lambda: gg.gg_fp8_forward(x, off, p, E, N, K, y=_normal(5, N + 8)),
            lambda: gg.gg_fp8_forward(x, off, p, E, N, K, workspace=torch.empty(8, device=DEV)),
            lambda: gg.gg_fp8_dgrad(x, off, p, E, N, K, activation="swiglu"),
            lambda: gg.gg_fp8_dgrad(x, off, p, E, N, K, h1=x, activation="swiglu"),     # needs halves
            lambda: gg.gg_fp8_dgrad(x, off, p, E, N, K, dh1_out=x),
            lambda: gg.fp8_experts(_normal(E, 2 * N, K), _normal(E, K, N + 8))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(gg.GGError):
        gg.gg_fp8_forward(x, off, p, E, N, K, y=x)                        # the output is the input
    with pytest.raises(ValueError):
        gg.fp8_experts(_normal(E, 2 * N, K).requires_grad_(True), _normal(E, K, N))


def test_the_other_layout_is_refused(made):
    gg, q, s, x, off = made
    p, t = gg.gg_fp8_pack(q, s), gg.gg_fp8_pack_transposed(q, s)
    assert p.numel() == t.numel()
    w = gg.fp8_experts(_normal(E, 2 * N, K), _normal(E, K, N))
    for call in (lambda: gg.gg_fp8_dgrad(x, off, p, E, N, K), lambda: gg.gg_fp8_forward(x, off, t, E, N, K),
                 lambda: gg.gg_fp8_forward(x[:, :56].contiguous(), off, p, E, N, 56),
                 lambda: gg.gg_fp8_forward(x, off, w.fc1, E, 2 * N, K),              # packed in halves
                 lambda: gg.gg_fp8_glu_forward(x, off, w.fc1_t, w.fc2, E, K, N),
                 lambda: gg.gg_fp8_glu_dgrad(x, _normal(5, 2 * N), off, w.fc1, w.fc2_t, E, K, N)):
        with pytest.raises(ValueError, match="holds"):
            call()
    y, _ = gg.gg_fp8_forward(x, off, p, E, N, K)
    t.copy_(p)                                                                       # written since
    assert bitwise_equal(gg.gg_fp8_forward(x, off, t, E, N, K)[0], y)
    assert bitwise_equal(gg.gg_fp8_forward(x, off, p.clone(), E, N, K)[0], y)


def _guarded(nbytes, tail=1 << 16):
    """(a byte buffer of nbytes, the guard behind it)."""
    t = torch.full((nbytes + tail,), 7, dtype=torch.uint8, device=DEV)
    return t[:nbytes], t[nbytes:]


@pytest.mark.parametrize("M", [13, 300, 4099])
def test_bad_offsets_stay_in_bounds(M):
    """Decreasing and out-of-range offsets: results are undefined, but nothing outside the buffers is touched and the
    calls return, forward and backward (streaming items that quantize, small tiles, pairs of rows)."""
    import moe_expert_grouped_ragged_amd as gg
    n, H, F = 3, 72, 144
    w = gg.fp8_experts(_normal(n, 2 * F, H), _normal(n, H, F))
    x, dy, h1 = _normal(M, H), _normal(M, H), _normal(M, 2 * F)
    bf = lambda t, width: t.view(torch.bfloat16).view(M, width)   # noqa: E731
    for off in ([0, M, 0, M], [-5, M + 80, 20, 10], [M, 0, M, 0], [1 << 40, 0, 3, -(1 << 40)], [M, M, 7, M],
                [M + 1, M + 1, M + 1, M + 1], [1 << 62, 1 << 62, 1 << 62, 1 << 62]):
        log(f"[fp8] M={M} offsets {off}")
        offd = torch.tensor(off, device=DEV)
        bufs = {k: _guarded(b) for k, b in (("y", M * H * 2), ("h1", M * F * 4), ("dx", M * H * 2), ("a", M * F * 2),
                                            ("dh", M * F * 4), ("f", gg.fp8_glu_workspace_bytes(M, H, F)),
                                            ("b", gg.fp8_glu_workspace_bytes(M, H, F, True)), ("w", gg.fp8_workspace_bytes(M, F)),
                                            ("v", gg.fp8_workspace_bytes(M, 2 * F, 2)))}
        b = {k: v[0] for k, v in bufs.items()}
        gg.gg_fp8_glu_forward(x, offd, w.fc1, w.fc2, n, H, F, h1_out=bf(b["h1"], 2 * F), y=bf(b["y"], H), workspace=b["f"])
        gg.gg_fp8_glu_dgrad(dy, h1, offd, w.fc1_t, w.fc2_t, n, H, F, dx=bf(b["dx"], H), workspace=b["b"])
        gg.gg_fp8_forward(h1, offd, w.fc2, n, H, F, activation="swiglu", a_out=bf(b["a"], F), y=bf(b["y"], H), workspace=b["w"])
        gg.gg_fp8_dgrad(bf(b["a"], F), offd, w.fc1_t, n, 2 * F, H, halves=2, h1=h1, activation="swiglu",
                        dh1_out=bf(b["dh"], 2 * F), dx=bf(b["dx"], H), workspace=b["v"])
        torch.cuda.synchronize()
        for k, (_, guard) in bufs.items():
            assert bool((guard == 7).all()), k


@pytest.mark.parametrize("E,M,K", [(1, 16, 264), (1, 17, 264), (8, 64, 264), (8, 65, 264), (4, 40, 4096), (4, 40, 4104), (2, 24, 8)])
def test_both_sides_of_the_small_batch_rules(E, M, K):
    """Rows quantized in the product and by a launch of their own, streamed and tiled: the same bits as in a batch where
    they are among many."""
    import moe_expert_grouped_ragged_amd as gg
    n = 136
    q, s = gg.gg_fp8_quantize_weights(_normal(E, n, K))
    packed = gg.gg_fp8_pack(q, s)
    x = _normal(M, K)
    off = torch.tensor([M * e // E for e in range(E + 1)], device=DEV)
    y, _ = gg.gg_fp8_forward(x, off, packed, E, n, K)
    many = x.repeat_interleave(40, 0)
    big, _ = gg.gg_fp8_forward(many, off * 40, packed, E, n, K)
    assert bitwise_equal(big[::40].contiguous(), y) and bitwise_equal(big[39::40].contiguous(), y)

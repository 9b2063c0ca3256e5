"""GPU: sums of more than 2048 columns, where a streaming item has 32 rows at most, so that an expert of a small batch
is several items, and of more than 4096, where no expert is streamed (products, and both epilogues of the gated
block), each bit for bit against calls that run otherwise."""
import numpy as np
import pytest
import torch

from gpu_harness import bitwise_equal

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _normal(shape, seed, size=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * size).to(torch.bfloat16)


def _off(counts, lead=0):
    return torch.from_numpy(np.concatenate([[lead], lead + np.cumsum(counts)]).astype(np.int64)).to(DEV)


@pytest.mark.parametrize("how", ["fp32", "scaled"])
@pytest.mark.parametrize("E,owner", [(1, 0), (8, 0), (8, 5), (9, 8)])      # one expert: a launch quantizes; from 8 on the product
@pytest.mark.parametrize("M", [33, 40, 63, 64])
@pytest.mark.parametrize("K", [2056, 4096])
def test_an_expert_of_several_streaming_items(K, M, E, owner, how):
    """All rows belong to one expert; as few rows at a time as one item, and among many rows in tiles, they are the same."""
    import moe_expert_grouped_ragged_amd as gg
    N = 392
    q, s = gg.gg_fp8_quantize_weights(_normal((E, N, K), 1, 0.02))
    t, ts = gg.gg_fp8_quantize_weights(_normal((E, K, N), 2, 0.02))
    fwd, back = gg.gg_fp8_pack(q, s), gg.gg_fp8_pack_transposed(t, ts)
    x = _normal((M, K), 3)
    many = torch.cat([x, _normal((600, K), 4)])
    for call in (lambda r, o: gg.gg_fp8_forward(r, o, fwd, E, N, K, sums=how)[0],
                 lambda r, o: gg.gg_fp8_dgrad(r, o, back, E, K, N, sums=how)[0]):
        def run(r):
            return call(r, _off([len(r) if e == owner else 0 for e in range(E)]))
        y = run(x)
        assert bitwise_equal(run(many)[:M], y)
        for lo in range(0, M, 17):
            assert bitwise_equal(run(x[lo:lo + 17].contiguous()), y[lo:lo + 17]), lo


@pytest.mark.parametrize("how", [None, "fp32", "scaled"])
@pytest.mark.parametrize("counts,F", [([1], 136), ([1, 0, 5, 2], 392), ([40, 0, 3, 21], 136), ([300, 0, 70, 129], 520), ([1500, 33, 1900], 2040)])
def test_the_block_where_nothing_is_streamed(counts, F, how):
    import moe_expert_grouped_ragged_amd as gg
    H, act, E = 4104, "swiglu", len(counts)
    off = _off(counts, 3)
    M = int(off[-1]) + 2
    live = slice(3, int(off[-1]))
    w = gg.fp8_experts(_normal((E, 2 * F, H), 5, H ** -0.5), _normal((E, H, F), 6, F ** -0.5))
    x, dy = _normal((M, H), 7), _normal((M, H), 8)
    h1, _ = gg.gg_fp8_forward(x, off, w.fc1, E, 2 * F, H, halves=2, sums=how)
    y, _ = gg.gg_fp8_forward(h1, off, w.fc2, E, H, F, activation=act, sums=how)
    da, _ = gg.gg_fp8_dgrad(dy, off, w.fc2_t, E, H, F, sums=how)
    dx, _ = gg.gg_fp8_dgrad(da, off, w.fc1_t, E, 2 * F, H, halves=2, h1=h1, activation=act, sums=how)
    by, bh, bx = (torch.full((M, width), 7.0, dtype=torch.bfloat16, device=DEV) for width in (H, 2 * F, H))
    gg.gg_fp8_glu_forward(x, off, w.fc1, w.fc2, E, H, F, activation=act, h1_out=bh, y=by, sums=how)
    gg.gg_fp8_glu_dgrad(dy, bh, off, w.fc1_t, w.fc2_t, E, H, F, activation=act, dx=bx, sums=how)
    y2, _ = gg.gg_fp8_glu_forward(x, off, w.fc1, w.fc2, E, H, F, activation=act, save_h1=False, sums=how)
    for name, got, want in (("h1", bh, h1), ("y", by, y), ("dx", bx, dx), ("y without h1", by, y2)):
        assert bitwise_equal(got[live], want[live]), name
        assert bool((got[:3] == 7).all()) and bool((got[-2:] == 7).all()), name

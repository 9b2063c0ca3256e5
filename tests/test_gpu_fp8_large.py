"""GPU: the block-scaled 8-bit products at the sizes where 256 x 256 and 128 x 256
tiles run (tests/host/fp8_driver.cpp holds the choice at these sizes).  A row's bits do not depend on the batch, so a large batch is compared bit for
bit with the same rows in calls of at most 64 rows (streaming items, held to
the 64-bit definition in test_gpu_fp8.py), and the gated block with its single
calls."""
import numpy as np
import pytest
import torch

from gpu_harness import bitwise_equal

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
# whole and partial tiles, experts without rows, streamed ones
MANY = [1024, 0, 257, 1, 352, 609, 96, 33, 511, 0, 128, 1085]    # tiles of 128 x 256
FEW = [1500, 33, 1900]                                           # tiles of 256 x 256


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _gg():
    import moe_expert_grouped_ragged_amd as gg
    return gg


def _normal(shape, seed, size=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * size).to(torch.bfloat16)


def _off(counts, lead=0):
    return torch.from_numpy(np.concatenate([[lead], lead + np.cumsum(counts)]).astype(np.int64)).to(DEV)


def _rows_one_by_one(call, x, off, width, E):
    """The same rows in batches of at most 64 of one expert each."""
    out = torch.empty(x.shape[0], width, dtype=torch.bfloat16, device=DEV)
    o = off.cpu().numpy()
    for e in range(E):
        for lo in range(int(o[e]), int(o[e + 1]), 64):
            hi = min(lo + 64, int(o[e + 1]))
            part = torch.zeros(E + 1, dtype=torch.int64, device=DEV)
            part[e + 1:] = hi - lo
            out[lo:hi] = call(x[lo:hi].contiguous(), part)
    return out


@pytest.mark.parametrize("counts", [MANY, FEW], ids=["many", "few"])
@pytest.mark.parametrize("N,K,halves", [(4096, 8, 1), (4088, 136, 1), (4096, 264, 1), (4128, 1032, 2), (3600, 640, 2)])
def test_forward_and_dgrad(counts, N, K, halves):
    gg = _gg()
    E, lead = len(counts), 5
    off = _off(counts, lead)
    M = int(off[-1]) + 7
    x = _normal((M, K), 1)
    q, s = gg.gg_fp8_quantize_weights(_normal((E, N, K), 2, 0.02), halves=halves)
    packed = gg.gg_fp8_pack(q, s, halves=halves)
    y = torch.full((M, N), 7.0, dtype=torch.bfloat16, device=DEV)
    gg.gg_fp8_forward(x, off, packed, E, N, K, halves=halves, y=y)
    want = _rows_one_by_one(lambda r, o: gg.gg_fp8_forward(r, o, packed, E, N, K, halves=halves)[0], x, off, N, E)
    live = slice(lead, int(off[-1]))
    assert bitwise_equal(y[live], want[live])
    assert bool((y[:lead] == 7).all()) and bool((y[-7:] == 7).all())
    # the transposed direction: K summed columns of N rows, as the weights [E, K, N] of the same numbers
    q, s = gg.gg_fp8_quantize_weights(_normal((E, K, N), 3, 0.02))
    packed = gg.gg_fp8_pack_transposed(q, s)
    dx = torch.full((M, N), 7.0, dtype=torch.bfloat16, device=DEV)
    gg.gg_fp8_dgrad(x, off, packed, E, K, N, dx=dx)
    want = _rows_one_by_one(lambda r, o: gg.gg_fp8_dgrad(r, o, packed, E, K, N)[0], x, off, N, E)
    assert bitwise_equal(dx[live], want[live]) and bool((dx[:lead] == 7).all()) and bool((dx[-7:] == 7).all())


@pytest.mark.parametrize("counts", [MANY + [2048, 513, 4096], FEW], ids=["many", "few"])
@pytest.mark.parametrize("H,F,act", [(264, 2048, "swiglu"), (136, 2040, "qgeglu"), (1032, 3968, "swiglu"), (8, 1928, "swiglu")])
def test_gated_block_is_its_single_calls(counts, H, F, act):
    gg = _gg()
    E = len(counts)
    off = _off(counts, 3)
    M = int(off[-1]) + 2
    live = slice(3, int(off[-1]))
    w = gg.fp8_experts(_normal((E, 2 * F, H), 4, H ** -0.5), _normal((E, H, F), 5, F ** -0.5))
    x, dy = _normal((M, H), 6), _normal((M, H), 7)
    h1, _ = gg.gg_fp8_forward(x, off, w.fc1, E, 2 * F, H, halves=2)
    y, _ = gg.gg_fp8_forward(h1, off, w.fc2, E, H, F, activation=act)
    da, _ = gg.gg_fp8_dgrad(dy, off, w.fc2_t, E, H, F)
    dx, _ = gg.gg_fp8_dgrad(da, off, w.fc1_t, E, 2 * F, H, halves=2, h1=h1, activation=act)
    for save in (True, False):
        bh = torch.full((M, 2 * F), 7.0, dtype=torch.bfloat16, device=DEV) if save else None
        by, _ = gg.gg_fp8_glu_forward(x, off, w.fc1, w.fc2, E, H, F, activation=act, save_h1=False, h1_out=bh)
        assert bitwise_equal(by[live], y[live]), save
        if save:
            assert bitwise_equal(bh[live], h1[live])
            assert bool((bh[:3] == 7).all()) and bool((bh[-2:] == 7).all())
    bx = gg.gg_fp8_glu_dgrad(dy, h1, off, w.fc1_t, w.fc2_t, E, H, F, activation=act)
    assert bitwise_equal(bx[live], dx[live])

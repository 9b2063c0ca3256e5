"""GPU: weights of more than 2^24 blocks are quantized (a grid of one dimension would pass 2^32 threads)."""
import pytest
import torch

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def test_more_blocks_than_one_grid_dimension_holds():
    import moe_expert_grouped_ragged_amd as gg
    E, N, K = 1024, 8, (1 << 21) + 8
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 80 GB of device memory")
    shape = gg.fp8_scale_shape(E, N, K)
    assert shape[0] * shape[1] * shape[2] > 1 << 24
    w = torch.zeros(E, N, K, dtype=torch.bfloat16, device=DEV)
    q = torch.full((E, N, K), 0x55, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
    # blocks at both ends, and around the 2^24th
    places = [(0, 0), (0, K - 1), (1, 130), (1023, 0), (1023, 128 * 16383 - 1), (1023, K - 1)]
    for i, (e, k) in enumerate(places):
        w[e, i % N, k] = 3.0 * 2.0 ** i
    got, s = gg.gg_fp8_quantize_weights(w, q=q)
    assert got is q
    s = s.view(torch.uint8)
    for i, (e, k) in enumerate(places):
        # 3 2^i = 384 * 2^(i - 7): the least power of two that keeps it below 448
        assert int(s[e, 0, k // 128]) == i - 7 + 127 and float(q[e, i % N, k].float()) == 384.0, (e, k)
        s[e, 0, k // 128] = 1
        q.view(torch.uint8)[e, i % N, k] = 0
    # all other blocks: zeros, of the least scale
    assert bool((s == 1).all())
    for e in range(0, E, 64):
        assert not q.view(torch.uint8)[e:e + 64].any()

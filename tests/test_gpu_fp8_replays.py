"""GPU: the gated block captured into a graph, replayed with other splits: each replay against the single calls
made eagerly for that split, so the two ways through the operators are held to each other at every split."""
import numpy as np
import pytest
import torch

import workload
from gpu_harness import bitwise_equal

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.mark.parametrize("how", [None, "fp32", "scaled"])
@pytest.mark.parametrize("counts0", [[300, 0, 70, 20, 0, 513, 33, 1], [5, 0, 9, 1, 0, 20, 0, 2]])
def test_replays_are_the_single_calls(counts0, how):
    import moe_expert_grouped_ragged_amd as gg
    c = workload.custom_case(counts0, 128, 96, seed=76)
    E, H, F, M = c.E, c.H, c.F, c.M
    w = gg.fp8_experts(c.w1.to(DEV), c.w2.to(DEV))
    x, dy = c.x.to(DEV), c.dy.to(DEV)
    off = torch.from_numpy(np.ascontiguousarray(c.offsets)).to(DEV)
    y, h1, dx = (torch.empty(M, n, dtype=torch.bfloat16, device=DEV) for n in (H, 2 * F, H))
    ws = torch.empty(max(gg.fp8_glu_workspace_bytes(M, H, F), gg.fp8_glu_workspace_bytes(M, H, F, True)), dtype=torch.uint8, device=DEV)

    def block():
        gg.gg_fp8_glu_forward(x, off, w.fc1, w.fc2, E, H, F, h1_out=h1, y=y, workspace=ws, sums=how)
        gg.gg_fp8_glu_dgrad(dy, h1, off, w.fc1_t, w.fc2_t, E, H, F, dx=dx, workspace=ws, sums=how)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block()
    rng = np.random.default_rng(6)
    for counts in (counts0, counts0[::-1], [M] + [0] * 7, [0] * 7 + [M], list(rng.multinomial(M, np.ones(E) / E))):
        off.copy_(torch.from_numpy(workload.offsets_from_counts(np.asarray(counts))).to(DEV))
        for t in (y, h1, dx):
            t.fill_(7.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        g1, _ = gg.gg_fp8_forward(x, off, w.fc1, E, 2 * F, H, halves=2, sums=how)
        gy, _ = gg.gg_fp8_forward(g1, off, w.fc2, E, H, F, activation="swiglu", sums=how)
        da, _ = gg.gg_fp8_dgrad(dy, off, w.fc2_t, E, H, F, sums=how)
        gx, _ = gg.gg_fp8_dgrad(da, off, w.fc1_t, E, 2 * F, H, halves=2, h1=g1, activation="swiglu", sums=how)
        for name, got, want in (("h1", h1, g1), ("y", y, gy), ("dx", dx, gx)):
            assert bitwise_equal(got, want), (counts, name)
            assert not torch.isnan(got).any() and not (got == 7).all(), (counts, name)

"""GPU: the 8-bit forward at batches large enough that the quantization takes
two rows at a time (16 rows for each CU onwards)."""
import pytest
import torch

from gpu_harness import log
from test_gpu_int8 import _rows, _weights

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _pairs_from():
    return 16 * torch.cuda.get_device_properties(0).multi_processor_count


def _guarded(nbytes, tail=1 << 16):
    """(a byte buffer of nbytes, the guard behind it)."""
    t = torch.full((nbytes + tail,), 7, dtype=torch.uint8, device=DEV)
    return t[:nbytes], t[nbytes:]


@pytest.mark.parametrize("act", [None, "swiglu"])
def test_experts_without_rows_touch_nothing(act):
    """Every expert empty, the common offset odd or even, inside the batch or at its end: no row of y, A or the
    workspace is written."""
    import moe_expert_grouped_ragged_amd as gg
    E, K, N = 3, 264, 40
    wq, ws = _weights(E, N, K, 3)
    packed = gg.gg_int8_pack(wq.to(DEV), ws.to(DEV))
    for M in (_pairs_from() + 1, _pairs_from() + 4):
        x = _rows(M, K if act is None else 2 * K, 5).to(DEV)
        for at in (0, 1, 4, 5, M - 1, M):
            log(f"[int8 pairs] {act} M={M} all offsets {at}")
            y, y_end = _guarded(M * N * 2)
            a, a_end = _guarded(M * K * 2)
            wsp, ws_end = _guarded(gg.int8_workspace_bytes(M, K))
            gg.gg_int8_forward(x, torch.full((E + 1,), at, device=DEV), packed, E, N, K, activation=act,
                               a_out=None if act is None else a.view(torch.bfloat16).view(M, K),
                               y=y.view(torch.bfloat16).view(M, N), workspace=wsp)
            torch.cuda.synchronize()
            for t in (y, y_end, a, a_end, wsp, ws_end):
                assert bool((t == 7).all())

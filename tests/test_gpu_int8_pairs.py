"""GPU: the 8-bit forward at batches large enough that the quantization takes
two rows at a time (16 rows for each CU onwards): against the definition in
64 bits, against the same rows taken one at a time, and at the edges of the
experts' rows; offsets that are wrong, below and above that size."""
import pytest
import torch

from gpu_harness import bitwise_equal, log
from test_gpu_int8 import _rows, _weights
from test_gpu_int8 import test_forward as _forward

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


# summed dimension: an odd number of 8-value units with padding behind (72, 264), a whole line of every lane (4096),
# and wider than a wave's registers (4104)
@pytest.mark.parametrize("K", [72, 264, 4096, 4104])
@pytest.mark.parametrize("act", [None, "swiglu", "qgeglu"])
@pytest.mark.parametrize("lead,tail", [(0, 0), (3, 2), (2, 1), (1, 0)])
def test_against_the_definition(K, act, lead, tail):
    """Odd and even first and last rows."""
    counts = [1500, 0, 1, 2047, 600 + _pairs_from() - 4096]
    assert lead + sum(counts) + tail >= _pairs_from()
    _forward(counts, K, 40, lead, tail, act)


@pytest.mark.parametrize("K", [72, 520, 4112])
@pytest.mark.parametrize("act", [None, "swiglu"])
def test_same_bits_as_one_row_at_a_time(K, act):
    """Rows of zeros, NaN and infinities in both places of a pair: what a row gives, it gives in small batches too,
    which take one row at a time."""
    import moe_expert_grouped_ragged_amd as gg
    M, N = _pairs_from() + 37, 40
    x = _rows(M, K if act is None else 2 * K, K)
    for i, v in ((10, 0.0), (21, 0.0), (32, float("nan")), (43, float("nan")), (54, float("inf")), (65, float("-inf")),
                 (76, 0.0), (77, float("nan")), (M - 1, float("nan"))):
        x[i, slice(None) if v == 0 else slice(K - 1, K)] = v
    x = x.to(DEV)
    wq, ws = _weights(1, N, K, 8)
    packed = gg.gg_int8_pack(wq.to(DEV), ws.to(DEV))

    def run(rows):
        n = rows.shape[0]
        return gg.gg_int8_forward(rows, torch.tensor([0, n], device=DEV), packed, 1, N, K, activation=act,
                                  save_a=act is not None)

    y, a = run(x)
    small = [run(x[lo:lo + 1000].contiguous()) for lo in range(0, M, 1000)]
    ys = torch.cat([t for t, _ in small])
    assert torch.equal(torch.isnan(y), torch.isnan(ys))
    assert bitwise_equal(torch.nan_to_num(y), torch.nan_to_num(ys))
    if act is not None:
        as_ = torch.cat([t for _, t in small])
        assert torch.equal(torch.isnan(a), torch.isnan(as_)) and bitwise_equal(torch.nan_to_num(a), torch.nan_to_num(as_))
    assert not bool(y[[10, 21, 76]].any())
    assert bool(torch.isnan(y[[32, 43, 54, 65, 77, M - 1]]).all())


@pytest.mark.parametrize("rows", ["one at a time", "pairs"])
@pytest.mark.parametrize("act", [None, "swiglu"])
def test_bad_offsets_stay_in_bounds(rows, act):
    """Decreasing and out-of-range offsets: results are undefined, but nothing outside the buffers is touched and
    the calls return, forward and backward."""
    import moe_expert_grouped_ragged_amd as gg
    E, K, N = 3, 72, 144
    M = 121 if rows == "one at a time" else _pairs_from() + 1
    wq, ws = _weights(E, N, K, 9)
    packed, packed_t = gg.gg_int8_pack(wq.to(DEV), ws.to(DEV)), gg.gg_int8_pack_transposed(wq.to(DEV), ws.to(DEV))
    x = _rows(M, K if act is None else 2 * K, 6).to(DEV)
    dy, h1 = _rows(M, N if act is None else N // 2, 7).to(DEV), None if act is None else _rows(M, N, 8).to(DEV)
    bf = lambda t, w: t.view(torch.bfloat16).view(M, w)   # noqa: E731
    for off in ([0, M, 0, M], [-5, M + 80, 20, 10], [M, 0, M, 0], [1 << 40, 0, 3, -(1 << 40)], [M, M, 7, M],
                [M + 1, M + 1, M + 1, M + 1], [1 << 62, 1 << 62, 1 << 62, 1 << 62]):
        log(f"[int8 pairs] {act} M={M} offsets {off}")
        offd = torch.tensor(off, device=DEV)
        y, y_end = _guarded(M * N * 2)
        a, a_end = _guarded(M * K * 2)
        w1, w1_end = _guarded(gg.int8_workspace_bytes(M, K))
        gg.gg_int8_forward(x, offd, packed, E, N, K, activation=act, a_out=None if act is None else bf(a, K), y=bf(y, N),
                           workspace=w1)
        dx, dx_end = _guarded(M * K * 2)
        dh, dh_end = _guarded(M * N * 2)
        w2, w2_end = _guarded(gg.int8_workspace_bytes(M, N))
        gg.gg_int8_dgrad(dy, offd, packed_t, E, N, K, h1=h1, activation=act, dh1_out=None if act is None else bf(dh, N),
                         dx=bf(dx, K), workspace=w2)
        torch.cuda.synchronize()
        for t in (y_end, a_end, w1_end, dx_end, dh_end, w2_end):
            assert bool((t == 7).all())

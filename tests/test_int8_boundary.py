"""The C boundary of the 8-bit expert products on the CPU: sizes, and bad
arguments rejected before any HIP call."""
import pytest


@pytest.fixture
def gg():
    import moe_expert_grouped_ragged_amd as gg
    return gg


P = 1 << 20   # 16-byte aligned stand-in addresses: every call below is refused before they are used


def test_sizes(gg):
    # rows to a multiple of 32, the summed dimension to one of 128, then E * pad128(N) scales
    assert gg.int8_packed_bytes(1, 8, 8) == 32 * 128 + 4 * 128
    assert gg.int8_packed_bytes(3, 40, 264) == 3 * (64 * 384 + 4 * 128)
    assert gg.int8_packed_bytes(3, 40, 264, transposed=True) == 3 * (288 * 128 + 4 * 128)
    assert gg.int8_packed_bytes(128, 4096, 4096) == 128 * (4096 * 4096 + 4 * 4096)
    for E, N, K in ((0, 8, 8), (1025, 8, 8), (1, 12, 8), (1, 8, 4), (1, 131080, 8), (1, 8, 131080), (1, 0, 8),
                    (1, 65536, 32768)):
        assert gg.int8_packed_bytes(E, N, K) == 0
    assert gg.int8_workspace_bytes(10, 264) == 10 * (384 + 4)
    assert gg.int8_workspace_bytes(0, 264) == 0 and gg.int8_workspace_bytes(1, 0) == 0


def test_forward_refusals(gg):
    L, INV, MIS, WS, ALI = (gg.lib, gg.GG_ERR_INVALID_ARGUMENT, gg.GG_ERR_MISALIGNED, gg.GG_ERR_WORKSPACE_TOO_SMALL,
                            gg.GG_ERR_ALIASING)
    big = 1 << 28

    def fwd(x=P, off=2 * P, M=16, w=4 * P, E=2, N=40, K=64, act=-1, a=None, ws=32 * P, wsb=big, y=600 * P):
        return L.gg_int8_forward(x, off, M, w, E, N, K, act, a, ws, wsb, y, None)

    for kw in ({"x": None}, {"off": None}, {"w": None}, {"ws": None}, {"y": None}, {"E": 0}, {"E": 1025}, {"N": 44},
               {"K": 60}, {"N": 0}, {"K": -8}, {"M": -1}, {"M": 1 << 31}, {"K": 131080}, {"act": 7},
               {"a": 700 * P}):          # A without an activation
        assert fwd(**kw) == INV, kw
    for kw in ({"x": P + 8}, {"w": 4 * P + 4}, {"ws": 32 * P + 8}, {"y": 600 * P + 2}, {"off": 2 * P + 4},
               {"act": 0, "a": 700 * P + 8}):
        assert fwd(**kw) == MIS, kw
    assert fwd(wsb=16 * (128 + 4) - 1) == WS
    for kw in ({"y": P}, {"y": 4 * P}, {"ws": P}, {"y": 32 * P}, {"act": 1, "a": P}, {"act": 1, "a": 600 * P}):
        assert fwd(**kw) == ALI, kw
    assert fwd(M=0, x=None, y=None, ws=None) == gg.GG_OK


def test_dgrad_refusals(gg):
    L, INV, MIS, WS, ALI = (gg.lib, gg.GG_ERR_INVALID_ARGUMENT, gg.GG_ERR_MISALIGNED, gg.GG_ERR_WORKSPACE_TOO_SMALL,
                            gg.GG_ERR_ALIASING)
    big = 1 << 28

    def dgr(dy=P, h1=None, off=2 * P, M=16, w=4 * P, E=2, N=48, K=64, act=-1, d=None, ws=32 * P, wsb=big, dx=600 * P):
        return L.gg_int8_dgrad(dy, h1, off, M, w, E, N, K, act, d, ws, wsb, dx, None)

    for kw in ({"dy": None}, {"off": None}, {"w": None}, {"ws": None}, {"dx": None}, {"act": 0}, {"h1": 700 * P},
               {"d": 700 * P}, {"act": 0, "h1": 700 * P, "N": 40}, {"act": 5, "h1": 700 * P}, {"N": 131088}):
        assert dgr(**kw) == INV, kw
    for kw in ({"dy": P + 8}, {"act": 0, "h1": 700 * P + 8}, {"act": 0, "h1": 700 * P, "d": 800 * P + 8},
               {"dx": 600 * P + 8}, {"off": 2 * P + 4}):
        assert dgr(**kw) == MIS, kw
    assert dgr(wsb=16 * (128 + 4) - 1) == WS
    for kw in ({"dx": P}, {"act": 0, "h1": 700 * P, "d": 700 * P}, {"act": 0, "h1": 700 * P, "d": P}, {"dx": 32 * P}):
        assert dgr(**kw) == ALI, kw
    assert dgr(M=0) == gg.GG_OK


def test_pack_and_quantize_refusals(gg):
    L, INV, MIS, WS, ALI = (gg.lib, gg.GG_ERR_INVALID_ARGUMENT, gg.GG_ERR_MISALIGNED, gg.GG_ERR_WORKSPACE_TOO_SMALL,
                            gg.GG_ERR_ALIASING)
    need = gg.int8_packed_bytes(2, 40, 64)
    assert L.gg_int8_pack(None, 2 * P, 2, 40, 64, 0, 4 * P, need, None) == INV
    assert L.gg_int8_pack(P, 2 * P, 2, 44, 64, 0, 4 * P, need, None) == INV
    assert L.gg_int8_pack(P, 2 * P, 2, 40, 64, 0, 4 * P + 8, need, None) == MIS
    assert L.gg_int8_pack(P, 2 * P, 2, 40, 64, 0, 4 * P, need - 1, None) == WS
    assert L.gg_int8_pack(P, 2 * P, 2, 40, 64, 0, P, need, None) == ALI
    assert L.gg_int8_quantize_rows(P, 4, 60, 4 * P, 8 * P, None) == INV
    assert L.gg_int8_quantize_rows(P, 4, 64, None, 8 * P, None) == INV
    assert L.gg_int8_quantize_rows(P + 8, 4, 64, 4 * P, 8 * P, None) == MIS
    assert L.gg_int8_quantize_rows(P, 4, 64, 4 * P + 4, 8 * P, None) == MIS
    assert L.gg_int8_quantize_rows(P, 4, 64, P + 64, 8 * P, None) == ALI
    assert L.gg_int8_quantize_rows(P, 0, 64, None, None, None) == gg.GG_OK

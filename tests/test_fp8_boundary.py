"""The C boundary of the block-scaled 8-bit products on the CPU: sizes, and bad
arguments rejected before any HIP call."""
import pytest


@pytest.fixture
def gg():
    import moe_expert_grouped_ragged_amd as gg
    return gg


P = 1 << 20   # 16-byte aligned stand-in addresses: every call below is refused before they are used
BIG = 1 << 28


def test_sizes(gg):
    # both dimensions to whole blocks; a byte of scale for each block, the summed dimension's in whole dwords
    assert gg.fp8_packed_bytes(1, 8, 8) == 128 * 128 + 4
    assert gg.fp8_packed_bytes(3, 40, 264) == 3 * (128 * 384 + 3 * 4)        # the transposed matrix has more scales
    assert gg.fp8_packed_bytes(2, 304, 264, 2) == 2 * (512 * 384 + 4 * 4)
    assert gg.fp8_packed_bytes(128, 4096, 4096) == 128 * (4096 * 4096 + 32 * 32)
    assert gg.lib.gg_fp8_scale_bytes(2, 304, 264, 2) == 2 * 4 * 3 and gg.fp8_scale_shape(2, 304, 264, 2) == (2, 4, 3)
    for E, N, K, h in ((0, 8, 8, 1), (1025, 8, 8, 1), (1, 12, 8, 1), (1, 8, 4, 1), (1, 1 << 22, 8, 1), (1, 8, 1 << 22, 1),
                       (1, 0, 8, 1), (1, 65536, 32768, 1), (1, 8, 8, 0), (1, 8, 8, 3), (1, 24, 8, 2)):
        assert gg.fp8_packed_bytes(E, N, K, h) == 0 and gg.lib.gg_fp8_scale_bytes(E, N, K, h) == 0
    assert gg.fp8_workspace_bytes(10, 264) == 10 * (384 + 4)
    assert gg.fp8_workspace_bytes(10, 304, 2) == 10 * (512 + 4) and gg.fp8_workspace_bytes(10, 640) == 10 * (640 + 8)
    assert gg.fp8_workspace_bytes(0, 264) == 0 and gg.fp8_workspace_bytes(1, 0) == 0
    assert gg.fp8_glu_workspace_bytes(0, 64, 40) == 0 and gg.fp8_glu_workspace_bytes(5, 64, 44) == 0
    assert gg.fp8_glu_workspace_bytes(5, 64, 40) > 0 and gg.fp8_glu_workspace_bytes(5, 64, 40, True) > 0


def test_forward_refusals(gg):
    L, INV, MIS, WS, ALI = (gg.lib, gg.GG_ERR_INVALID_ARGUMENT, gg.GG_ERR_MISALIGNED, gg.GG_ERR_WORKSPACE_TOO_SMALL,
                            gg.GG_ERR_ALIASING)

    def fwd(x=P, off=2 * P, M=16, w=4 * P, E=2, N=48, K=64, halves=1, act=-1, a=None, ws=32 * P, wsb=BIG, y=600 * P):
        return L.gg_fp8_forward(x, off, M, w, E, N, K, halves, act, a, ws, wsb, y, None)

    for kw in ({"x": None}, {"off": None}, {"w": None}, {"ws": None}, {"y": None}, {"E": 0}, {"E": 1025}, {"N": 44},
               {"K": 60}, {"N": 0}, {"K": -8}, {"M": -1}, {"M": 1 << 31}, {"K": 1 << 22}, {"act": 7}, {"halves": 0},
               {"halves": 3}, {"halves": 2, "N": 40}, {"a": 700 * P}):
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

    def dgr(dy=P, h1=None, off=2 * P, M=16, w=4 * P, E=2, N=48, K=64, halves=2, act=-1, d=None, ws=32 * P, wsb=BIG, dx=600 * P):
        return L.gg_fp8_dgrad(dy, h1, off, M, w, E, N, K, halves, act, d, ws, wsb, dx, None)

    for kw in ({"dy": None}, {"off": None}, {"w": None}, {"ws": None}, {"dx": None}, {"act": 0}, {"h1": 700 * P},
               {"d": 700 * P}, {"act": 0, "h1": 700 * P, "halves": 1}, {"act": 5, "h1": 700 * P}, {"N": 40}):
        assert dgr(**kw) == INV, kw
    for kw in ({"dy": P + 8}, {"act": 0, "h1": 700 * P + 8}, {"act": 0, "h1": 700 * P, "d": 800 * P + 8},
               {"dx": 600 * P + 8}, {"off": 2 * P + 4}):
        assert dgr(**kw) == MIS, kw
    assert dgr(wsb=16 * (256 + 4) - 1) == WS
    for kw in ({"dx": P}, {"act": 0, "h1": 700 * P, "d": 700 * P}, {"act": 0, "h1": 700 * P, "d": P}, {"dx": 32 * P}):
        assert dgr(**kw) == ALI, kw
    assert dgr(M=0) == gg.GG_OK


def test_pack_and_quantize_refusals(gg):
    L, INV, MIS, WS, ALI = (gg.lib, gg.GG_ERR_INVALID_ARGUMENT, gg.GG_ERR_MISALIGNED, gg.GG_ERR_WORKSPACE_TOO_SMALL,
                            gg.GG_ERR_ALIASING)
    need = gg.fp8_packed_bytes(2, 48, 64)
    assert L.gg_fp8_pack(None, 2 * P, 2, 48, 64, 1, 0, 4 * P, need, None) == INV
    assert L.gg_fp8_pack(P, 2 * P, 2, 44, 64, 1, 0, 4 * P, need, None) == INV
    assert L.gg_fp8_pack(P, 2 * P, 2, 48, 64, 1, 0, 4 * P + 8, need, None) == MIS
    assert L.gg_fp8_pack(P + 4, 2 * P, 2, 48, 64, 1, 0, 4 * P, need, None) == MIS
    assert L.gg_fp8_pack(P, 2 * P, 2, 48, 64, 1, 1, 4 * P, need - 1, None) == WS
    assert L.gg_fp8_pack(P, 2 * P, 2, 48, 64, 1, 0, P, need, None) == ALI
    assert L.gg_fp8_quantize_weights(P, 2, 48, 60, 1, 4 * P, 8 * P, None) == INV
    assert L.gg_fp8_quantize_weights(P, 2, 48, 64, 1, None, 8 * P, None) == INV
    assert L.gg_fp8_quantize_weights(P, 2, 48, 64, 1, 4 * P, None, None) == INV
    assert L.gg_fp8_quantize_weights(P + 8, 2, 48, 64, 1, 4 * P, 8 * P, None) == MIS
    assert L.gg_fp8_quantize_weights(P, 2, 48, 64, 1, 4 * P + 4, 8 * P, None) == MIS
    assert L.gg_fp8_quantize_weights(P, 2, 48, 64, 1, P + 64, 8 * P, None) == ALI


def test_block_refusals(gg):
    L, INV, MIS, WS, ALI = (gg.lib, gg.GG_ERR_INVALID_ARGUMENT, gg.GG_ERR_MISALIGNED, gg.GG_ERR_WORKSPACE_TOO_SMALL,
                            gg.GG_ERR_ALIASING)

    def fwd(x=P, off=2 * P, M=16, fc1=4 * P, fc2=8 * P, E=2, H=64, F=40, act=0, ws=32 * P, wsb=BIG, h1=None, y=600 * P):
        return L.gg_fp8_glu_forward(x, off, M, fc1, fc2, E, H, F, act, ws, wsb, h1, y, None)

    for kw in ({"x": None}, {"off": None}, {"fc1": None}, {"fc2": None}, {"ws": None}, {"y": None}, {"E": 0}, {"H": 60},
               {"F": 44}, {"F": 0}, {"M": -1}, {"act": -1}, {"act": 2}):
        assert fwd(**kw) == INV, kw
    for kw in ({"x": P + 8}, {"fc1": 4 * P + 8}, {"fc2": 8 * P + 8}, {"ws": 32 * P + 8}, {"y": 600 * P + 8}, {"h1": 700 * P + 8},
               {"off": 2 * P + 4}):
        assert fwd(**kw) == MIS, kw
    assert fwd(wsb=gg.fp8_glu_workspace_bytes(16, 64, 40) - 1) == WS
    for kw in ({"y": P}, {"y": 4 * P}, {"y": 8 * P}, {"h1": P}, {"h1": 600 * P}, {"ws": 4 * P}):
        assert fwd(**kw) == ALI, kw
    assert fwd(M=0, x=None) == gg.GG_OK

    def dgr(dy=P, h1=700 * P, off=2 * P, M=16, fc1=4 * P, fc2=8 * P, E=2, H=64, F=40, act=0, ws=32 * P, wsb=BIG, dx=600 * P):
        return L.gg_fp8_glu_dgrad(dy, h1, off, M, fc1, fc2, E, H, F, act, ws, wsb, dx, None)

    for kw in ({"dy": None}, {"h1": None}, {"off": None}, {"fc1": None}, {"fc2": None}, {"ws": None}, {"dx": None}, {"act": -1}):
        assert dgr(**kw) == INV, kw
    for kw in ({"dy": P + 8}, {"h1": 700 * P + 8}, {"fc1": 4 * P + 8}, {"fc2": 8 * P + 8}, {"dx": 600 * P + 8}):
        assert dgr(**kw) == MIS, kw
    assert dgr(wsb=gg.fp8_glu_workspace_bytes(16, 64, 40, True) - 1) == WS
    for kw in ({"dx": P}, {"dx": 700 * P}, {"dx": 4 * P}, {"ws": P}):
        assert dgr(**kw) == ALI, kw
    assert dgr(M=0) == gg.GG_OK

"""The C boundary of the expert adapters on the CPU: sizes, and bad arguments
rejected before any HIP call."""
import pytest

P = 1 << 24   # 16-byte aligned stand-in addresses: every call below is refused before they are used


@pytest.fixture
def gg():
    import moe_expert_grouped_ragged_amd as gg
    return gg


def test_workspace(gg):
    # 32-row blocks: du parts (fp32, one chunk of 1024 columns), du (bf16, 32 wide), du transposed (3 x bf16);
    # 100 rows of 3 experts make at most 100 // 32 + 3 blocks, and no expert has more than 256 rows
    assert gg.adapter_workspace_bytes(100, 3, 64, 64, 16) == 6 * 32 * (16 * 4 + 32 * 2 + 16 * 6)
    assert gg.adapter_workspace_bytes(0, 3, 64, 64, 16) == 0
    for M, E, N, K, r in ((8, 0, 64, 64, 8), (8, 1, 60, 64, 8), (8, 1, 64, 4, 8), (8, 1, 64, 64, 0), (8, 1, 64, 64, 65)):
        assert gg.adapter_workspace_bytes(M, E, N, K, r) == 0


def test_forward_refusals(gg):
    INV, MIS, ALI = gg.GG_ERR_INVALID_ARGUMENT, gg.GG_ERR_MISALIGNED, gg.GG_ERR_ALIASING

    def fwd(x=P, off=2 * P, M=16, a=3 * P, b=4 * P, E=2, N=40, K=64, r=6, base=5 * P, u=6 * P, y=7 * P):
        return gg.lib.gg_adapter_forward(x, off, M, a, b, E, N, K, r, 1.0, base, u, y, None)

    for kw in ({"x": None}, {"off": None}, {"a": None}, {"b": None}, {"u": None}, {"y": None}, {"E": 0}, {"E": 1025},
               {"N": 44}, {"K": 60}, {"N": 1 << 22}, {"M": -1}, {"M": 1 << 31}, {"r": 0}, {"r": 65}):
        assert fwd(**kw) == INV, kw
    for kw in ({"x": P + 8}, {"a": 3 * P + 2}, {"b": 4 * P + 2}, {"u": 6 * P + 2}, {"y": 7 * P + 8}, {"base": 5 * P + 8},
               {"off": 2 * P + 4}):
        assert fwd(**kw) == MIS, kw
    for kw in ({"y": P}, {"u": P}, {"y": 6 * P}, {"y": 3 * P}, {"y": 5 * P + 16}, {"u": 5 * P}):
        assert fwd(**kw) == ALI, kw
    assert fwd(M=0, x=None, y=None, u=None) == gg.GG_OK


def test_backward_refusals(gg):
    INV, MIS, WS, ALI = (gg.GG_ERR_INVALID_ARGUMENT, gg.GG_ERR_MISALIGNED, gg.GG_ERR_WORKSPACE_TOO_SMALL,
                         gg.GG_ERR_ALIASING)
    need = gg.adapter_workspace_bytes(16, 2, 40, 64, 6)

    def bwd(dy=P, x=2 * P, u=3 * P, off=4 * P, M=16, a=5 * P, b=6 * P, E=2, N=40, K=64, r=6, base=7 * P, ws=8 * P,
            wsb=need, dx=10 * P, da=11 * P, db=12 * P):
        return gg.lib.gg_adapter_backward(dy, x, u, off, M, a, b, E, N, K, r, 1.0, base, ws, wsb, dx, da, db, 0, None)

    for kw in ({"dy": None}, {"x": None}, {"u": None}, {"off": None}, {"a": None}, {"b": None}, {"ws": None}, {"dx": None},
               {"da": None}, {"db": None}, {"r": 65}, {"K": 4}, {"M": 1 << 31}):
        assert bwd(**kw) == INV, kw
    for kw in ({"dy": P + 8}, {"u": 3 * P + 2}, {"ws": 8 * P + 8}, {"dx": 10 * P + 8}, {"da": 11 * P + 4},
               {"db": 12 * P + 4}, {"base": 7 * P + 8}, {"off": 4 * P + 4}):
        assert bwd(**kw) == MIS, kw
    assert bwd(wsb=need - 1) == WS
    for kw in ({"dx": P}, {"dx": 2 * P}, {"dx": 7 * P + 16}, {"da": 8 * P}, {"db": 11 * P}, {"ws": 3 * P}, {"da": 5 * P}):
        assert bwd(**kw) == ALI, kw

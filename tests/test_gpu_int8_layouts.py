"""GPU: a packed buffer given to the call that needs the other layout is refused,
where the sizes alone would let it pass; what was written since, copies and views
are taken as they are."""
import pytest
import torch

from gpu_harness import bitwise_equal
from test_gpu_int8 import _rows, _weights

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
E, N = 2, 64


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


@pytest.fixture
def made():
    import moe_expert_grouped_ragged_amd as gg
    wq, ws = (t.to(DEV) for t in _weights(E, N, N, 1))
    return gg, wq, ws, _rows(5, N, 2).to(DEV), torch.tensor([0, 2, 5], device=DEV)


def test_the_other_layout_is_refused(made):
    gg, wq, ws, x, off = made
    p, t = gg.gg_int8_pack(wq, ws), gg.gg_int8_pack_transposed(wq, ws)
    assert p.numel() == t.numel()
    for call in (lambda: gg.gg_int8_dgrad(x, off, p, E, N, N), lambda: gg.gg_int8_forward(x, off, t, E, N, N),
                 lambda: gg.gg_int8_forward(x, off[:2].contiguous(), p, 1, N, N),        # other experts
                 lambda: gg.gg_int8_forward(x[:, :56].contiguous(), off, p, E, N, 56)):  # another summed dimension
        with pytest.raises(ValueError, match="packed holds"):
            call()
    w = gg.int8_experts(*(torch.ones(s, dtype=torch.bfloat16, device=DEV) for s in ((E, 2 * N, N), (E, N, N))))
    with pytest.raises(ValueError, match="packed holds"):
        gg.gg_int8_forward(x, off, w.fc2_t, E, N, N)


def test_what_changed_since_is_taken(made):
    gg, wq, ws, x, off = made
    p, t = gg.gg_int8_pack(wq, ws), gg.gg_int8_pack_transposed(wq, ws)
    y, _ = gg.gg_int8_forward(x, off, p, E, N, N)
    dx, _ = gg.gg_int8_dgrad(x, off, t, E, N, N)
    again = gg.gg_int8_pack(wq, ws)
    assert gg.gg_int8_pack_transposed(wq, ws, packed=again) is again           # packed anew
    assert bitwise_equal(gg.gg_int8_dgrad(x, off, again, E, N, N)[0], dx)
    gg.gg_int8_pack(wq, ws, packed=again[:])                                   # through a view
    assert bitwise_equal(gg.gg_int8_forward(x, off, again, E, N, N)[0], y)
    again.copy_(t)                                                             # written otherwise
    assert bitwise_equal(gg.gg_int8_dgrad(x, off, again, E, N, N)[0], dx)
    for same in (p.clone(), p[:], p.view(torch.int8)):
        assert bitwise_equal(gg.gg_int8_forward(x, off, same, E, N, N)[0], y)
    with torch.inference_mode():
        q = gg.gg_int8_pack(wq, ws)
        assert bitwise_equal(gg.gg_int8_forward(x, off, q, E, N, N)[0], y)

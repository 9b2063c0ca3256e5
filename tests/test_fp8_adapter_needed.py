"""Fp8AdapterExpertMLP's and Fp8ExpertMLP's backward make what is asked for, on
the CPU: the operators are replaced by recorders, so this sees the calls, not
their results."""
import pytest
import torch

E, H, F, R, M = 2, 16, 24, 4, 5


def _bf(*s):
    return torch.ones(*s, dtype=torch.bfloat16)


@pytest.fixture
def gg(monkeypatch):
    import moe_expert_grouped_ragged_amd as gg
    calls = []

    def fp8_forward(x, offsets, packed, E, N, K, halves=1, activation=None, save_a=False, **kw):
        assert halves == (2 if packed == "fc1" else 1)
        return _bf(x.shape[0], N), _bf(x.shape[0], K) if save_a else None

    def fp8_dgrad(dy, offsets, packed, E, N, K, halves=1, h1=None, activation=None):
        assert halves == (2 if packed == "fc1_t" else 1)
        calls.append(packed)
        return _bf(dy.shape[0], K), None if h1 is None else _bf(dy.shape[0], N)

    def adapter_forward(x, offsets, a, b, scale, base=None, y=None):
        return _bf(x.shape[0], b.shape[1]), _bf(x.shape[0], a.shape[1])

    def adapter_backward(dy, x, u, offsets, a, b, scale, base=None, dx=None):
        calls.append("adapter of " + ("fc2" if b.shape[1] == H else "fc1") + ("" if base is None else " on the base"))
        return _bf(x.shape[0], x.shape[1]), torch.ones(a.shape), torch.ones(b.shape)

    def glu_forward(x, offsets, fc1, fc2, E, H, F, activation, save_h1):
        calls.append("h1 saved" if save_h1 else "h1 not saved")
        return _bf(x.shape[0], H), _bf(x.shape[0], 2 * F) if save_h1 else None

    def glu_dgrad(dy, h1, offsets, fc1_t, fc2_t, E, H, F, activation):
        calls.append((fc1_t, fc2_t, dy.is_contiguous()))
        return _bf(dy.shape[0], H)

    for name, fake in (("gg_fp8_forward", fp8_forward), ("gg_fp8_dgrad", fp8_dgrad), ("gg_adapter_forward", adapter_forward),
                       ("gg_adapter_backward", adapter_backward), ("gg_fp8_glu_forward", glu_forward),
                       ("gg_fp8_glu_dgrad", glu_dgrad)):
        monkeypatch.setattr(gg, name, fake)
    gg.test_calls = calls
    yield gg
    del gg.test_calls


FC2, FC1 = ["fc2_t", "adapter of fc2 on the base"], ["fc1_t", "adapter of fc1 on the base"]


@pytest.mark.parametrize("needed,calls", [
    (("x", "a1", "b1", "a2", "b2"), FC2 + FC1),
    (("a1", "b1", "a2", "b2"), FC2 + FC1),
    (("x",), FC2 + FC1),
    (("b1",), FC2 + FC1),
    (("a2", "b2"), ["adapter of fc2"]),          # nothing below FC2 is asked for
])
def test_only_what_is_needed(gg, needed, calls):
    t = {n: torch.ones(*s, dtype=torch.bfloat16).requires_grad_(n in needed)
         for n, s in (("x", (M, H)), ("a1", (E, R, H)), ("b1", (E, 2 * F, R)), ("a2", (E, R, F)), ("b2", (E, H, R)))}
    w = gg.Fp8Experts(E, H, F, "fc1", "fc2", "fc1_t", "fc2_t")
    y = gg.Fp8AdapterExpertMLP.apply(t["x"], torch.zeros(E + 1, dtype=torch.int64), w, t["a1"], t["b1"], t["a2"], t["b2"], 0.5)
    y.backward(torch.ones_like(y))
    assert gg.test_calls == calls
    for n, v in t.items():
        assert (v.grad is not None) == (n in needed), n
        if v.grad is not None:
            assert v.grad.dtype == torch.bfloat16 and v.grad.shape == v.shape


def test_block(gg):
    w = gg.Fp8Experts(E, H, F, "fc1", "fc2", "fc1_t", "fc2_t")
    x = _bf(M, H)
    off = torch.zeros(E + 1, dtype=torch.int64)
    gg.Fp8ExpertMLP.apply(x, off, w)
    assert gg.test_calls == ["h1 not saved"]
    x.requires_grad_(True)
    gg.Fp8ExpertMLP.apply(x, off, w).backward(torch.ones(H, M, dtype=torch.bfloat16).t())
    assert gg.test_calls[1:] == ["h1 saved", ("fc1_t", "fc2_t", True)] and x.grad.shape == x.shape

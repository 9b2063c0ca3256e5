"""Int8AdapterExpertMLP's backward makes what is asked for, on the CPU: the
operators are replaced by recorders, so this sees the calls, not their results."""
import pytest
import torch

E, H, F, R, M = 2, 16, 24, 4, 5


@pytest.fixture
def gg(monkeypatch):
    import moe_expert_grouped_ragged_amd as gg
    calls = []
    bf = lambda *s: torch.ones(*s, dtype=torch.bfloat16)   # noqa: E731

    def int8_forward(x, offsets, packed, E, N, K, activation=None, save_a=False, **kw):
        return bf(x.shape[0], N), bf(x.shape[0], K) if save_a else None

    def adapter_forward(x, offsets, a, b, scale, base=None, y=None):
        return bf(x.shape[0], b.shape[1]), bf(x.shape[0], a.shape[1])

    def int8_dgrad(dy, offsets, packed, E, N, K, h1=None, activation=None):
        calls.append(packed)
        return bf(dy.shape[0], K), None if h1 is None else bf(dy.shape[0], N)

    def adapter_backward(dy, x, u, offsets, a, b, scale, base=None, dx=None):
        calls.append("adapter of " + ("fc2" if b.shape[1] == H else "fc1") + ("" if base is None else " on the base"))
        return bf(x.shape[0], x.shape[1]), torch.ones(a.shape), torch.ones(b.shape)

    for name, fake in (("gg_int8_forward", int8_forward), ("gg_adapter_forward", adapter_forward),
                       ("gg_int8_dgrad", int8_dgrad), ("gg_adapter_backward", adapter_backward)):
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
    (("b2",), ["adapter of fc2"]),
])
def test_only_what_is_needed(gg, needed, calls):
    t = {n: torch.ones(*s, dtype=torch.bfloat16).requires_grad_(n in needed)
         for n, s in (("x", (M, H)), ("a1", (E, R, H)), ("b1", (E, 2 * F, R)), ("a2", (E, R, F)), ("b2", (E, H, R)))}
    w = gg.Int8Experts(E, H, F, "fc1", "fc2", "fc1_t", "fc2_t")
    y = gg.Int8AdapterExpertMLP.apply(t["x"], torch.zeros(E + 1, dtype=torch.int64), w, t["a1"], t["b1"], t["a2"], t["b2"], 0.5)
    y.backward(torch.ones_like(y))
    assert gg.test_calls == calls
    for n, v in t.items():
        assert (v.grad is not None) == (n in needed), n
        if v.grad is not None:
            assert v.grad.dtype == torch.bfloat16 and v.grad.shape == v.shape

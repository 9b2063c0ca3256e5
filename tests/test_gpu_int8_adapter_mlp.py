"""GPU: the 8-bit expert MLP with adapters (Int8AdapterExpertMLP): its output and
gradients against the same network in 64 bits on the CPU, fed the values the
operators round where they are defined to; the operators inside a HIP graph
with changing offsets; the example."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import workload
from gpu_harness import bitwise_equal, log

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _setup(counts, H, F, r, seed):
    import moe_expert_grouped_ragged_amd as gg
    c = workload.custom_case(counts, H, F, seed=seed)
    g = torch.Generator().manual_seed(seed)
    E = c.E
    ad = [(torch.randn(s, generator=g) * 0.1).to(torch.bfloat16)
          for s in ((E, r, H), (E, 2 * F, r), (E, r, F), (E, H, r))]
    return gg, c, ad, torch.from_numpy(np.ascontiguousarray(c.offsets)).to(DEV)


@pytest.mark.parametrize("act", ["swiglu", "qgeglu"])
def test_wrapper_is_the_explicit_calls(act):
    gg, c, ad, off = _setup([40, 0, 300, 7], 128, 96, 12, 61)
    E, H, F = c.E, c.H, c.F
    w = gg.int8_experts(c.w1.to(DEV), c.w2.to(DEV))
    x = c.x.to(DEV).requires_grad_(True)
    p = [t.to(DEV).requires_grad_(True) for t in ad]
    y = gg.Int8AdapterExpertMLP.apply(x, off, w, *p, 0.5, act)
    y.backward(c.dy.to(DEV))
    a1, b1, a2, b2 = (t.detach() for t in p)
    xd, dy = x.detach(), c.dy.to(DEV)
    h0, _ = gg.gg_int8_forward(xd, off, w.fc1, E, 2 * F, H)
    h1, u1 = gg.gg_adapter_forward(xd, off, a1, b1, 0.5, base=h0)
    y0, a = gg.gg_int8_forward(h1, off, w.fc2, E, H, F, activation=act, save_a=True)
    yr, u2 = gg.gg_adapter_forward(a, off, a2, b2, 0.5, base=y0)
    da0, _ = gg.gg_int8_dgrad(dy, off, w.fc2_t, E, H, F)
    da, ga2, gb2 = gg.gg_adapter_backward(dy, a, u2, off, a2, b2, 0.5, base=da0)
    dx0, dh1 = gg.gg_int8_dgrad(da, off, w.fc1_t, E, 2 * F, H, h1=h1, activation=act)
    dx, ga1, gb1 = gg.gg_adapter_backward(dh1, xd, u1, off, a1, b1, 0.5, base=dx0)
    assert bitwise_equal(y.detach(), yr) and bitwise_equal(x.grad, dx)
    for t, g in zip(p, (ga1, gb1, ga2, gb2)):
        assert bitwise_equal(t.grad, g.to(torch.bfloat16))


def test_mlp_against_64_bits():
    """The whole network in 64 bits without any rounding.  Quantizing a row
    errs by top / 127 / sqrt(12) = top / 440 of its values' scale: 0.7 % for normals
    (top about 3 of 64 .. 256 values), 1.4 % for A and dH1, products of two (top about 6).
    Y: x and W1 make 1.0 % of H1, both factors of A carry it (1.6 %), then A itself
    (1.4 %) and W2 (0.6 %): 2.2 % together.  dX: dY and W2 1.0 %, the derivative at H1
    about as much, dH1 1.4 %, W1 0.7 %: 2.1 %.  The adapters' gradients hold parts of
    these, and the bf16 roundings (0.2 %) change none.  4 % is nearly twice the sums."""
    gg, c, ad, off = _setup([40, 0, 200, 7], 256, 64, 8, 62)
    w = gg.int8_experts(c.w1.to(DEV), c.w2.to(DEV))
    x = c.x.to(DEV).requires_grad_(True)
    p = [t.to(DEV).requires_grad_(True) for t in ad]
    y = gg.Int8AdapterExpertMLP.apply(x, off, w, *p, 0.5)
    y.backward(c.dy.to(DEV))
    xr = c.x.double().requires_grad_(True)
    pr = [t.double().requires_grad_(True) for t in ad]
    outs = []
    for e in range(c.E):
        xe = xr[int(c.offsets[e]):int(c.offsets[e + 1])]
        h = xe @ c.w1[e].double().T + 0.5 * (xe @ pr[0][e].T) @ pr[1][e].T
        gate, up = h[:, :c.F], h[:, c.F:]
        a = gate * torch.sigmoid(gate) * up
        outs.append(a @ c.w2[e].double().T + 0.5 * (a @ pr[2][e].T) @ pr[3][e].T)
    yr = torch.cat(outs)
    yr.backward(c.dy.double())
    for name, got, want in [("y", y, yr), ("dx", x.grad, xr.grad)] + [
            (n, t.grad, r.grad) for n, t, r in zip(("a1", "b1", "a2", "b2"), p, pr)]:
        rel = float((got.detach().cpu().double() - want.detach()).norm() / want.detach().norm())
        log(f"[int8 mlp] {name}: {rel:.4f}")
        assert rel <= 0.04, (name, rel)
        assert not torch.isnan(got).any()


def test_graph_replays_follow_new_offsets():
    """Every call of a training step captured once, replayed with other splits,
    eager work and synchronization in between; each replay bit for bit the eager result."""
    counts0 = [300, 0, 70, 20, 0, 513, 33, 1]
    gg, c, ad, off = _setup(counts0, 128, 96, 12, 63)
    E, H, F, M = c.E, c.H, c.F, c.M
    w = gg.int8_experts(c.w1.to(DEV), c.w2.to(DEV))
    a1, b1, a2, b2 = (t.to(DEV) for t in ad)
    x, dy = c.x.to(DEV), c.dy.to(DEV)
    new = lambda n, dt=torch.bfloat16: torch.empty(M, n, dtype=dt, device=DEV)   # noqa: E731

    def buffers():
        return {"h1": new(2 * F), "u1": new(12), "a": new(F), "u2": new(12), "y": new(H), "da": new(F), "dh1": new(2 * F),
                "dx": new(H), "ga1": torch.empty(E, 12, H, device=DEV), "gb1": torch.empty(E, 2 * F, 12, device=DEV),
                "ga2": torch.empty(E, 12, F, device=DEV), "gb2": torch.empty(E, H, 12, device=DEV)}

    ws = torch.empty(max(gg.int8_workspace_bytes(M, max(2 * F, H)), gg.adapter_workspace_bytes(M, E, 2 * F, H, 12),
                         gg.adapter_workspace_bytes(M, E, H, F, 12)), dtype=torch.uint8, device=DEV)

    def step(o, b):
        gg.gg_int8_forward(x, o, w.fc1, E, 2 * F, H, y=b["h1"], workspace=ws)
        gg.gg_adapter_forward(x, o, a1, b1, 0.5, base=b["h1"], y=b["h1"], u=b["u1"])
        gg.gg_int8_forward(b["h1"], o, w.fc2, E, H, F, activation="swiglu", a_out=b["a"], y=b["y"], workspace=ws)
        gg.gg_adapter_forward(b["a"], o, a2, b2, 0.5, base=b["y"], y=b["y"], u=b["u2"])
        gg.gg_int8_dgrad(dy, o, w.fc2_t, E, H, F, dx=b["da"], workspace=ws)
        gg.gg_adapter_backward(dy, b["a"], b["u2"], o, a2, b2, 0.5, base=b["da"], dx=b["da"], da=b["ga2"], db=b["gb2"],
                               workspace=ws)
        gg.gg_int8_dgrad(b["da"], o, w.fc1_t, E, 2 * F, H, h1=b["h1"], activation="swiglu", dh1_out=b["dh1"], dx=b["dx"],
                         workspace=ws)
        gg.gg_adapter_backward(b["dh1"], x, b["u1"], o, a1, b1, 0.5, base=b["dx"], dx=b["dx"], da=b["ga1"], db=b["gb1"],
                               workspace=ws)

    bufs = buffers()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(off, bufs)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(off, bufs)
    torch.cuda.synchronize()
    rng = np.random.default_rng(5)
    for counts in (counts0, counts0[::-1], [M] + [0] * 7, [0] * 7 + [M], list(rng.multinomial(M, np.ones(E) / E)), counts0):
        log(f"[int8 mlp] replay {counts}")
        o = torch.from_numpy(workload.offsets_from_counts(np.asarray(counts))).to(DEV)
        off.copy_(o)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = {k: v.clone() for k, v in bufs.items()}
        ref = {k: torch.full_like(v, 7.0) for k, v in bufs.items()}
        step(o, ref)
        torch.cuda.synchronize()
        for k in got:
            assert torch.equal(got[k].view(torch.uint8), ref[k].view(torch.uint8)), k


def test_example_learns_and_serves():
    spec = importlib.util.spec_from_file_location("example", os.path.join(ROOT, "examples", "int8_adapter_experts.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    losses, token, batch = m.main(steps=20)
    log(f"[int8 mlp] example losses {losses[0]:.4f} .. {losses[-1]:.4f}")
    assert all(np.isfinite(losses)) and losses[-1] < losses[0]
    # the same row in another batch: fp32 sums of the adapters may split otherwise, one bf16 step of the largest value
    assert float((token.float() - batch.float()).abs().max()) <= 2.0 ** -7 * float(batch.float().abs().max())


def test_no_rows():
    """A batch without rows: an empty output, an empty input gradient, zero adapter gradients."""
    gg, c, ad, _ = _setup([3, 0], 64, 32, 4, 64)
    w = gg.int8_experts(c.w1.to(DEV), c.w2.to(DEV))
    x = torch.empty(0, 64, dtype=torch.bfloat16, device=DEV, requires_grad=True)
    p = [t.to(DEV).requires_grad_(True) for t in ad]
    off = torch.zeros(3, dtype=torch.int64, device=DEV)
    y = gg.Int8AdapterExpertMLP.apply(x, off, w, *p, 0.5)
    y.backward(torch.empty_like(y))
    assert y.shape == (0, 64) and x.grad.shape == (0, 64)
    assert all(torch.count_nonzero(t.grad) == 0 for t in p)


def test_refusals():
    gg, c, ad, off = _setup([3, 5], 64, 32, 4, 65)
    w1, w2 = c.w1.to(DEV), c.w2.to(DEV)
    for a, b in ((w1.clone().requires_grad_(True), w2), (w1[:, :-8], w2), (w1[0], w2), (w1, w2[:1])):
        with pytest.raises(ValueError):
            gg.int8_experts(a, b)
    w = gg.int8_experts(w1, w2)
    x, p = c.x.to(DEV), [t.to(DEV) for t in ad]
    for i, bad in ((0, p[0].float()), (1, p[1][:, :-8]), (2, p[2][:1]), (3, p[3].cpu())):
        q = list(p)
        q[i] = bad
        with pytest.raises(ValueError):
            gg.Int8AdapterExpertMLP.apply(x, off, w, *q, 0.5)
    with pytest.raises(ValueError):
        gg.Int8AdapterExpertMLP.apply(x[:, :-8], off, w, *p, 0.5)
    with pytest.raises(ValueError):
        gg.Int8AdapterExpertMLP.apply(x, off, w, *p, 0.5, "relu")


def test_outputs_allocated_for_a_given_stream():
    """Memory that is free for the current stream, but whose last reader is still queued on it, is not given to a
    call on another stream: the reader's copy keeps its value."""
    gg, c, ad, off = _setup([40, 0, 30, 7], 512, 256, 8, 66)
    x, w = c.x.to(DEV), gg.int8_experts(c.w1.to(DEV), c.w2.to(DEV))
    st = torch.cuda.Stream()
    want, _ = gg.gg_int8_forward(x, off, w.fc1, c.E, 512, 512)
    busy = torch.ones(4096, 4096, device=DEV)
    torch.cuda.synchronize()
    for _ in range(4):
        busy = busy @ busy * 2.0 ** -12                       # keeps the current stream busy
    old = torch.full((c.M, 512), 2.0, dtype=torch.bfloat16, device=DEV)
    copy = old.clone()                                        # reads `old`, later
    del old
    y, _ = gg.gg_int8_forward(x, off, w.fc1, c.E, 512, 512, stream=st)
    st.synchronize()
    torch.cuda.synchronize()
    assert bitwise_equal(y, want) and bool((copy == 2.0).all())

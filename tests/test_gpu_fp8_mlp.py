"""GPU: the gated block and the adapter MLP over 8-bit floating-point weights
(Fp8ExpertMLP, Fp8AdapterExpertMLP): outputs and gradients against the explicit
calls and against the same network in 64 bits on the CPU; a training step
inside a HIP graph with changing offsets; calls on another stream."""
import numpy as np
import pytest
import torch

import workload
from gpu_harness import bitwise_equal, log

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


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
def test_block_wrapper_is_the_explicit_calls(act):
    gg, c, _, off = _setup([40, 0, 300, 7], 128, 96, 4, 71)
    w = gg.fp8_experts(c.w1.to(DEV), c.w2.to(DEV))
    x = c.x.to(DEV).requires_grad_(True)
    y = gg.Fp8ExpertMLP.apply(x, off, w, act)
    dy = c.dy.to(DEV)
    y.backward(dy.t().contiguous().t())          # a gradient of other strides
    yr, h1 = gg.gg_fp8_glu_forward(x.detach(), off, w.fc1, w.fc2, c.E, c.H, c.F, activation=act)
    dx = gg.gg_fp8_glu_dgrad(dy, h1, off, w.fc1_t, w.fc2_t, c.E, c.H, c.F, activation=act)
    assert bitwise_equal(y.detach(), yr) and bitwise_equal(x.grad, dx)
    with torch.no_grad():
        assert bitwise_equal(gg.Fp8ExpertMLP.apply(x, off, w, act), yr)


@pytest.mark.parametrize("act", ["swiglu", "qgeglu"])
def test_adapter_wrapper_is_the_explicit_calls(act):
    gg, c, ad, off = _setup([40, 0, 300, 7], 128, 104, 12, 72)
    E, H, F = c.E, c.H, c.F
    w = gg.fp8_experts(c.w1.to(DEV), c.w2.to(DEV))
    x = c.x.to(DEV).requires_grad_(True)
    p = [t.to(DEV).requires_grad_(True) for t in ad]
    y = gg.Fp8AdapterExpertMLP.apply(x, off, w, *p, 0.5, act)
    y.backward(c.dy.to(DEV))
    a1, b1, a2, b2 = (t.detach() for t in p)
    xd, dy = x.detach(), c.dy.to(DEV)
    h0, _ = gg.gg_fp8_forward(xd, off, w.fc1, E, 2 * F, H, halves=2)
    h1, u1 = gg.gg_adapter_forward(xd, off, a1, b1, 0.5, base=h0)
    y0, a = gg.gg_fp8_forward(h1, off, w.fc2, E, H, F, activation=act, save_a=True)
    yr, u2 = gg.gg_adapter_forward(a, off, a2, b2, 0.5, base=y0)
    da0, _ = gg.gg_fp8_dgrad(dy, off, w.fc2_t, E, H, F)
    da, ga2, gb2 = gg.gg_adapter_backward(dy, a, u2, off, a2, b2, 0.5, base=da0)
    dx0, dh1 = gg.gg_fp8_dgrad(da, off, w.fc1_t, E, 2 * F, H, halves=2, h1=h1, activation=act)
    dx, ga1, gb1 = gg.gg_adapter_backward(dh1, xd, u1, off, a1, b1, 0.5, base=dx0)
    assert bitwise_equal(y.detach(), yr) and bitwise_equal(x.grad, dx)
    for t, g in zip(p, (ga1, gb1, ga2, gb2)):
        assert bitwise_equal(t.grad, g.to(torch.bfloat16))


@pytest.mark.parametrize("adapters", [False, True])
def test_mlp_against_64_bits(adapters):
    """The whole network in 64 bits without any rounding.  A value rounded to four
    significant bits errs by up to half a step of 1/8 of its power of two, evenly: 2^-4 / sqrt(3) / m for a
    value m in [1, 2), 2.7 % of it in the mean square for evenly spread log m.  Y: x and W1 make
    3.8 % of H1, both factors of A carry it (5.3 %), then A itself and W2 (2.7 % each): 6.5 %
    together.  dX: dY and W2 3.8 %, the derivative at H1 about as much (5.3 %), dH1 and W1: 6.5 %.
    The adapters' gradients hold parts of these, and the bf16 roundings (0.2 %) change
    none.  12 % is nearly twice the sums."""
    gg, c, ad, off = _setup([40, 0, 200, 7], 256, 64, 8, 73)
    w = gg.fp8_experts(c.w1.to(DEV), c.w2.to(DEV))
    x = c.x.to(DEV).requires_grad_(True)
    p = [t.to(DEV).requires_grad_(True) for t in ad]
    y = gg.Fp8AdapterExpertMLP.apply(x, off, w, *p, 0.5) if adapters else gg.Fp8ExpertMLP.apply(x, off, w)
    y.backward(c.dy.to(DEV))
    xr = c.x.double().requires_grad_(True)
    pr = [t.double().requires_grad_(True) for t in ad]
    outs, s = [], 0.5 if adapters else 0.0
    for e in range(c.E):
        xe = xr[int(c.offsets[e]):int(c.offsets[e + 1])]
        h = xe @ c.w1[e].double().T + s * (xe @ pr[0][e].T) @ pr[1][e].T
        gate, up = h[:, :c.F], h[:, c.F:]
        a = gate * torch.sigmoid(gate) * up
        outs.append(a @ c.w2[e].double().T + s * (a @ pr[2][e].T) @ pr[3][e].T)
    yr = torch.cat(outs)
    yr.backward(c.dy.double())
    pairs = [("y", y, yr), ("dx", x.grad, xr.grad)]
    if adapters:
        pairs += [(n, t.grad, r.grad) for n, t, r in zip(("a1", "b1", "a2", "b2"), p, pr)]
    for name, got, want in pairs:
        rel = float((got.detach().cpu().double() - want.detach()).norm() / want.detach().norm())
        log(f"[fp8 mlp] {name}: {rel:.4f}")
        assert rel <= 0.12, (name, rel)
        assert not torch.isnan(got).any()


@pytest.mark.parametrize("counts0", [[300, 0, 70, 20, 0, 513, 33, 1], [5, 0, 9, 1, 0, 20, 0, 2]])
def test_graph_replays_follow_new_offsets(counts0):
    """Every call of a step captured once, in two graphs that share a workspace, replayed with other splits, eager work
    and synchronization in between; each replay bit for bit the eager result."""
    gg, c, ad, off = _setup(counts0, 128, 96, 12, 74)
    E, H, F, M = c.E, c.H, c.F, c.M
    w = gg.fp8_experts(c.w1.to(DEV), c.w2.to(DEV))
    a1, b1 = ad[0].to(DEV), ad[1].to(DEV)
    x, dy = c.x.to(DEV), c.dy.to(DEV)
    new = lambda n: torch.empty(M, n, dtype=torch.bfloat16, device=DEV)   # noqa: E731

    def buffers():
        return {"h1": new(2 * F), "y": new(H), "dx": new(H), "k1": new(2 * F), "u1": new(12), "a": new(F), "z": new(H),
                "da": new(F), "dh1": new(2 * F), "dz": new(H)}

    ws = torch.empty(max(gg.fp8_glu_workspace_bytes(M, H, F), gg.fp8_glu_workspace_bytes(M, H, F, True),
                         gg.fp8_workspace_bytes(M, H), gg.fp8_workspace_bytes(M, 2 * F, 2), gg.fp8_workspace_bytes(M, F)),
                     dtype=torch.uint8, device=DEV)

    def block(o, b):
        gg.gg_fp8_glu_forward(x, o, w.fc1, w.fc2, E, H, F, h1_out=b["h1"], y=b["y"], workspace=ws)
        gg.gg_fp8_glu_dgrad(dy, b["h1"], o, w.fc1_t, w.fc2_t, E, H, F, dx=b["dx"], workspace=ws)

    def single(o, b):
        gg.gg_fp8_forward(x, o, w.fc1, E, 2 * F, H, halves=2, y=b["k1"], workspace=ws)
        gg.gg_adapter_forward(x, o, a1, b1, 0.5, base=b["k1"], y=b["k1"], u=b["u1"])
        gg.gg_fp8_forward(b["k1"], o, w.fc2, E, H, F, activation="swiglu", a_out=b["a"], y=b["z"], workspace=ws)
        gg.gg_fp8_dgrad(dy, o, w.fc2_t, E, H, F, dx=b["da"], workspace=ws)
        gg.gg_fp8_dgrad(b["da"], o, w.fc1_t, E, 2 * F, H, halves=2, h1=b["k1"], activation="swiglu", dh1_out=b["dh1"],
                        dx=b["dz"], workspace=ws)

    off_dev, bufs = off.clone(), buffers()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block(off_dev, bufs)
        single(off_dev, bufs)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graphs = []
    for step in (block, single):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(off_dev, bufs)
        graphs.append(graph)
    rng = np.random.default_rng(5)
    for counts in (counts0, counts0[::-1], [M] + [0] * 7, [0] * 7 + [M], list(rng.multinomial(M, np.ones(E) / E))):
        o = torch.from_numpy(workload.offsets_from_counts(np.asarray(counts))).to(DEV)
        off_dev.copy_(o)
        torch.cuda.synchronize()
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        got = {k: v.clone() for k, v in bufs.items()}
        want = {k: torch.full_like(v, 7.0) for k, v in bufs.items()}
        block(o, want)
        single(o, want)
        torch.cuda.synchronize()
        for k in got:
            assert bitwise_equal(got[k], want[k]), (counts, k)
        assert bitwise_equal(got["dx"], got["dx"]) and not torch.isnan(got["dx"]).any()


def test_another_stream():
    """Calls given a stream: their inputs are made on it, and nothing of theirs is used on another before it is waited for."""
    gg, c, _, off = _setup([40, 0, 300, 7], 128, 96, 4, 75)
    E, H, F = c.E, c.H, c.F
    w = gg.fp8_experts(c.w1.to(DEV), c.w2.to(DEV))
    want, h1 = gg.gg_fp8_glu_forward(c.x.to(DEV), off, w.fc1, w.fc2, E, H, F)
    dwant = gg.gg_fp8_glu_dgrad(c.dy.to(DEV), h1, off, w.fc1_t, w.fc2_t, E, H, F)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        x, dy = c.x.to(DEV), c.dy.to(DEV)
        q1, q2 = gg.gg_fp8_quantize_weights(c.w1.to(DEV), halves=2), gg.gg_fp8_quantize_weights(c.w2.to(DEV))
    for _ in range(3):
        fc1, fc2 = gg.gg_fp8_pack(*q1, halves=2, stream=s), gg.gg_fp8_pack(*q2, stream=s)
        t1, t2 = gg.gg_fp8_pack_transposed(*q1, halves=2, stream=s), gg.gg_fp8_pack_transposed(*q2, stream=s)
        y, h = gg.gg_fp8_glu_forward(x, off, fc1, fc2, E, H, F, stream=s)
        dx = gg.gg_fp8_glu_dgrad(dy, h, off, t1, t2, E, H, F, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        assert bitwise_equal(y, want) and bitwise_equal(dx, dwant)

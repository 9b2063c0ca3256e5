"""The operators around the frozen experts, as cases to measure: the expert
products over an 8-bit copy of the frozen weights (forward and input gradient,
with the activation fused into the token quantization) and the per-expert
low-rank adapters (forward, and the gradients of adapter weights and input).

``run`` computes a case with elementary torch operations in 32 bits
(``own = False``) or with the package's entry points (``own = True``);
``exact`` is the definition in 64 bits.

Definitions, for an expert e that owns rows [offsets[e], offsets[e+1]):

  quantization of a row v      s = max|v| / 127,  q = rint(127 v / max|v|) (0 for a zero row)
  int8_forward                 y = s * ws_e[n] * sum_k q[k] wq_e[n, k]
                               v = x, or v = A = bf16(act(gate) * up) of x = H1 = [gate | up]
  int8_dgrad                   v = ws_e[n] * g[n],  dx = s * sum_n q[n] wq_e[n, k]
                               g = dy, or g = dH1 = bf16(the activation's derivative at H1, times dA = dy)
  adapter_forward              u = x a_e^T,  y = base + scale * u b_e^T
  adapter_backward             du = scale * dy b_e,  dx = base + du a_e,
                               da_e = du^T x,  db_e = scale * dy^T u
"""
import math
import random

import numpy as np
import torch

own = False

SLOPE = {"swiglu": 1.0, "qgeglu": 1.702}
ADAPTER_SCALE = 0.5
PAD = 256            # rows of a padded expert block


def _case(name, op, E, rows, routing, K, N, act="none", save=False, r=0):
    return {"name": name, "op": op, "E": E, "rows": rows, "routing": routing, "K": K, "N": N, "act": act,
            "save": save, "r": r}


def listed():
    return [
        # one token of a decode step, sent to 8 of 128 experts: latency and the bytes of eight weight matrices
        _case("int8_token", "int8_forward", 128, 8, "tokens", 4096, 4096),
        # a small serving batch, about 24 rows for each expert: FC1 of the small-batch workload
        _case("int8_smallbatch", "int8_forward", 128, 2880, "uniform", 2688, 3712),
        # a training batch with Zipf-distributed expert sizes: FC2 with the activation in front, A saved
        _case("int8_zipf_glu", "int8_forward", 128, 131072, "zipf", 768, 2048, act="swiglu", save=True),
        # the largest workload's FC1: every expert padded to a multiple of 256 rows with zero rows
        _case("int8_padded", "int8_forward", 128, 262144, "padded", 4096, 4096),
        # a handful of experts with odd sizes, serving: QuickGeGLU in front of FC2, nothing saved
        _case("int8_odd_glu", "int8_forward", 5, 777, "uniform", 1048, 2056, act="qgeglu"),
        # input gradient of a small batch through FC2
        _case("int8_dgrad_smallbatch", "int8_dgrad", 128, 2880, "uniform", 1856, 2688),
        # input gradient of FC1 with the activation's derivative in front: the 32-expert workload
        _case("int8_dgrad_glu", "int8_dgrad", 32, 32768, "uniform", 2048, 1536, act="swiglu", save=True),
        # one token's adapters next to the frozen product
        _case("adapter_token", "adapter_forward", 128, 8, "tokens", 4096, 4096, r=16),
        # a small batch with a small odd rank
        _case("adapter_smallbatch", "adapter_forward", 128, 2880, "uniform", 2688, 3712, r=12),
        # adapter training, the largest workload
        _case("adapter_padded", "adapter_forward", 128, 262144, "padded", 4096, 4096, r=32),
        _case("adapter_bwd_uniform", "adapter_backward", 32, 32768, "uniform", 2048, 1536, r=16),
        _case("adapter_bwd_padded", "adapter_backward", 128, 262144, "padded", 2048, 4096, r=64),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case with sizes spread over the listed ones' ranges: one row to 131072, widths that
    are any multiples of 8, any number of experts, ranks that are no multiple of anything."""
    op = rng.choice(["int8_forward", "int8_forward", "int8_dgrad", "adapter_forward", "adapter_backward"])
    while True:
        rows = _spread(rng, 1, 131072)
        K, N = 8 * _spread(rng, 32, 512), 8 * _spread(rng, 32, 512)
        if 3072 not in (rows, K, N):
            break
    E = _spread(rng, 1, 128)
    routing = rng.choice(["uniform", "zipf", "padded" if rows >= PAD else "uniform"])
    if routing == "padded":
        rows = rows // PAD * PAD
    act, save, r = "none", False, 0
    if op.startswith("int8"):
        act = rng.choice(["none", "swiglu", "qgeglu"])
        if op == "int8_dgrad" and act != "none":
            N = 2 * max(64, N // 16 * 8)
            while N == 3072:
                N += 16
            save = True
        elif act != "none":
            save = rng.random() < 0.5
    else:
        r = _spread(rng, 2, 64)
    c = _case("", op, E, rows, routing, K, N, act, save, r)
    del c["name"]
    return c


def _probabilities(case, rank):
    p = 1.0 / (1.0 + rank) ** 1.2 if case["routing"] == "zipf" else np.ones(case["E"])
    return p / p.sum()


def _expected_experts(case):
    """Expected number of experts that own rows."""
    E, rows = case["E"], case["rows"]
    if case["routing"] == "tokens":
        return min(E, rows)
    p = _probabilities(case, np.arange(E))
    return float((1.0 - (1.0 - p) ** (rows // PAD if case["routing"] == "padded" else rows)).sum())


def _counts(case, seed):
    """(rows of each expert, rows of each that are real): they differ where blocks are padded."""
    r = np.random.RandomState(seed % (1 << 31))
    E, rows = case["E"], case["rows"]
    if case["routing"] == "tokens":          # one token's distinct experts
        c = np.zeros(E, np.int64)
        c[r.permutation(E)[:rows]] = 1
        return c, c
    p = _probabilities(case, r.permutation(E))
    if case["routing"] == "padded":
        c = r.multinomial(rows // PAD, p).astype(np.int64) * PAD
        return c, np.maximum(c - r.randint(0, PAD, E), 0)
    c = r.multinomial(rows, p).astype(np.int64)
    return c, c


def _normal(shape, std, gen):
    """N(0, std^2) in bf16, made in pieces."""
    out = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
    flat = out.view(-1)
    for at in range(0, flat.numel(), 1 << 27):
        n = min(1 << 27, flat.numel() - at)
        flat[at:at + n] = torch.randn(n, generator=gen, device="cuda").mul_(std).to(torch.bfloat16)
    return out


def _int8_weights(E, N, K, gen):
    """Frozen weights quantized for each output channel: (int8 [E, N, K], float32 [E, N])."""
    wq = torch.empty(E, N, K, dtype=torch.int8, device="cuda")
    ws = torch.empty(E, N, dtype=torch.float32, device="cuda")
    for e in range(E):
        w = torch.randn(N, K, generator=gen, device="cuda").mul_(0.02).to(torch.bfloat16).float()
        top = w.abs().amax(1)
        wq[e] = torch.round(w * 127 / top[:, None]).to(torch.int8)
        ws[e] = top / 127
    return wq, ws


def _inputs(case, seed):
    """Everything a pass reads, from the seed alone."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    E, M, K, N, op = case["E"], case["rows"], case["K"], case["N"], case["op"]
    counts, real = _counts(case, seed)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    live = torch.zeros(M, 1, device="cuda")
    at = torch.arange(M, device="cuda")
    owner = torch.from_numpy(np.repeat(np.arange(E), counts)).cuda()
    live[at < torch.from_numpy(offsets[:-1] + real).cuda()[owner]] = 1.0
    size = torch.exp(0.5 * torch.randn(M, 1, generator=gen, device="cuda")) * live   # tokens differ in scale

    def rows(width, std=1.0):
        t = _normal((M, width), std, gen)
        for lo in range(0, M, 1 << 14):
            t[lo:lo + (1 << 14)] *= size[lo:lo + (1 << 14)].to(torch.bfloat16)
        return t

    s = {"case": case, "offsets": torch.from_numpy(offsets).cuda(),
         "segments": [(e, int(offsets[e]), int(offsets[e + 1])) for e in range(E) if counts[e]]}
    if op == "int8_forward":
        s["x"] = rows(K if case["act"] == "none" else 2 * K)
        s["wq"], s["ws"] = _int8_weights(E, N, K, gen)
    elif op == "int8_dgrad":
        s["dy"] = rows(N if case["act"] == "none" else N // 2)
        s["h1"] = None if case["act"] == "none" else rows(N)
        s["wq"], s["ws"] = _int8_weights(E, N, K, gen)
    else:
        r = case["r"]
        s["x"] = rows(K)
        s["a"] = _normal((E, r, K), 1.0 / math.sqrt(K), gen)
        s["b"] = _normal((E, N, r), 0.5 / math.sqrt(r), gen)
        if op == "adapter_forward":
            s["base"] = rows(N)
        else:
            s["dy"], s["u"], s["base"] = rows(N), rows(r), rows(K)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own and case["op"].startswith("int8"):
        # the laid-out frozen weights that a program keeps
        import moe_expert_grouped_ragged_amd as gg
        pack = gg.gg_int8_pack if case["op"] == "int8_forward" else gg.gg_int8_pack_transposed
        s["packed"] = pack(s["wq"], s["ws"])
    return s


def _own(s):
    import moe_expert_grouped_ragged_amd as gg
    c = s["case"]
    E, K, N, op = c["E"], c["K"], c["N"], c["op"]
    act = None if c["act"] == "none" else c["act"]
    if op == "int8_forward":
        y, a = gg.gg_int8_forward(s["x"], s["offsets"], s["packed"], E, N, K, activation=act, save_a=c["save"])
        return {"y": y, "a": a} if c["save"] else {"y": y}
    if op == "int8_dgrad":
        dx, dh1 = gg.gg_int8_dgrad(s["dy"], s["offsets"], s["packed"], E, N, K, h1=s["h1"], activation=act)
        return {"dx": dx, "dh1": dh1} if act else {"dx": dx}
    if op == "adapter_forward":
        y, u = gg.gg_adapter_forward(s["x"], s["offsets"], s["a"], s["b"], ADAPTER_SCALE, base=s["base"])
        return {"y": y, "u": u}
    dx, da, db = gg.gg_adapter_backward(s["dy"], s["x"], s["u"], s["offsets"], s["a"], s["b"], ADAPTER_SCALE,
                                        base=s["base"])
    return {"dx": dx, "da": da, "db": db}


def _quantized(v):
    """(q as float32, s) of float32 rows."""
    top = v.abs().amax(1, keepdim=True)
    q = torch.round(v * 127 / torch.where(top > 0, top, 1.0))
    return q, top / 127


def run(s):
    if own:
        return _own(s)
    # A loop over the experts that own rows: their row counts differ, and one product padded
    # to the largest would do many times the work.
    c = s["case"]
    M, K, N, op = c["rows"], c["K"], c["N"], c["op"]
    if op == "int8_forward":
        y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
        a = s["x"]
        if c["act"] != "none":
            g, u = s["x"][:, :K].float(), s["x"][:, K:].float()
            a = (g * torch.sigmoid(SLOPE[c["act"]] * g) * u).to(torch.bfloat16)
        for e, lo, hi in s["segments"]:
            q, t = _quantized(a[lo:hi].float())
            y[lo:hi] = (q @ s["wq"][e].float().T * t * s["ws"][e]).to(torch.bfloat16)
        return {"y": y, "a": a} if c["save"] else {"y": y}
    if op == "int8_dgrad":
        dx = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
        g = s["dy"]
        if c["act"] != "none":
            k = SLOPE[c["act"]]
            d = s["dy"].float()
            gate, up = s["h1"][:, :N // 2].float(), s["h1"][:, N // 2:].float()
            sg = torch.sigmoid(k * gate)
            g = torch.cat([d * up * sg * (1 + k * gate * (1 - sg)), d * gate * sg], 1).to(torch.bfloat16)
        for e, lo, hi in s["segments"]:
            q, t = _quantized(g[lo:hi].float() * s["ws"][e])
            dx[lo:hi] = (q @ s["wq"][e].float() * t).to(torch.bfloat16)
        return {"dx": dx, "dh1": g} if c["act"] != "none" else {"dx": dx}
    a, b = s["a"], s["b"]
    if op == "adapter_forward":
        y, u = torch.empty_like(s["base"]), torch.empty(M, c["r"], dtype=torch.bfloat16, device="cuda")
        for e, lo, hi in s["segments"]:
            t = s["x"][lo:hi].float() @ a[e].float().T
            u[lo:hi] = t.to(torch.bfloat16)
            y[lo:hi] = (s["base"][lo:hi].float() + ADAPTER_SCALE * (t @ b[e].float().T)).to(torch.bfloat16)
        return {"y": y, "u": u}
    dx = torch.empty_like(s["base"])
    da, db = torch.zeros(a.shape, device="cuda"), torch.zeros(b.shape, device="cuda")
    for e, lo, hi in s["segments"]:
        d = s["dy"][lo:hi].float()
        du = ADAPTER_SCALE * (d @ b[e].float())
        dx[lo:hi] = (s["base"][lo:hi].float() + du @ a[e].float()).to(torch.bfloat16)
        da[e] = du.T @ s["x"][lo:hi].float()
        db[e] = ADAPTER_SCALE * (d.T @ s["u"][lo:hi].float())
    return {"dx": dx, "da": da, "db": db}


def work(case):
    M, K, N, E, r = case["rows"], case["K"], case["N"], case["E"], case["r"]
    hit = _expected_experts(case)
    glu = case["act"] != "none"
    if case["op"] == "int8_forward":
        read = M * K * (4 if glu else 2) + hit * N * (K + 4)
        return {"bytes": read + M * N * 2 + (M * K * 2 if case["save"] else 0), "flops": 2.0 * M * N * K}
    if case["op"] == "int8_dgrad":
        read = M * N * (3 if glu else 2) + hit * N * (K + 4)
        return {"bytes": read + M * K * 2 + (M * N * 2 if glu else 0), "flops": 2.0 * M * N * K}
    weights = hit * r * (K + N)
    if case["op"] == "adapter_forward":
        return {"bytes": M * (K + 2 * N + r) * 2 + weights * 2, "flops": 2.0 * M * r * (K + N)}
    return {"bytes": M * (3 * K + N + r) * 2 + weights * 2 + E * r * (K + N) * 4,
            "flops": 4.0 * M * r * (K + N)}


def exact(case, seed):
    s = _inputs(case, seed)
    M, K, N, op = case["rows"], case["K"], case["N"], case["op"]

    def empty(width):
        return torch.empty(M, width, dtype=torch.float64, device="cuda")

    def levels(v):
        top = torch.amax(torch.abs(v), 1, keepdim=True)
        return torch.nan_to_num(torch.round(torch.div(127 * v, top)), nan=0.0), top / 127.0

    # The operators round A and dH1 to bf16 where they are defined, before they are quantized.
    k = SLOPE.get(case["act"], 0.0)
    saved = empty(K if op == "int8_forward" else N) if case["act"] != "none" else None
    out = empty(N if op in ("int8_forward", "adapter_forward") else K)
    more = {}
    if op == "adapter_forward":
        more["u"] = empty(case["r"])
    if op == "adapter_backward":
        more["da"] = torch.zeros(s["a"].shape, dtype=torch.float64, device="cuda")
        more["db"] = torch.zeros(s["b"].shape, dtype=torch.float64, device="cuda")
    for e, lo, hi in s["segments"]:
        if op.startswith("int8"):
            w, ws = s["wq"][e].double(), s["ws"][e].double()
            if op == "int8_forward":
                v = s["x"][lo:hi].double()
                if saved is not None:
                    gate, up = v[:, :K], v[:, K:]
                    saved[lo:hi] = gate / (1.0 + torch.exp(-k * gate)) * up
                    v = saved[lo:hi].to(torch.bfloat16).double()
                q, t = levels(v)
                out[lo:hi] = torch.mm(q, w.t().contiguous()) * t * ws
            else:
                v = s["dy"][lo:hi].double()
                if saved is not None:
                    h = s["h1"][lo:hi].double()
                    gate, up = h[:, :N // 2], h[:, N // 2:]
                    z = torch.exp(-k * gate)
                    saved[lo:hi, :N // 2] = v * up * (1.0 + z + k * gate * z) / (1.0 + z) ** 2
                    saved[lo:hi, N // 2:] = v * gate / (1.0 + z)
                    v = saved[lo:hi].to(torch.bfloat16).double()
                q, t = levels(v * ws)
                out[lo:hi] = torch.mm(q, w) * t
            continue
        x, a, b = s["x"][lo:hi].double(), s["a"][e].double(), s["b"][e].double()
        if op == "adapter_forward":
            more["u"][lo:hi] = torch.mm(x, a.t())
            out[lo:hi] = s["base"][lo:hi].double() + torch.mm(more["u"][lo:hi], b.t()) * ADAPTER_SCALE
        else:
            dy = s["dy"][lo:hi].double()
            du = torch.mm(dy, b) * ADAPTER_SCALE
            out[lo:hi] = s["base"][lo:hi].double() + torch.mm(du, a)
            more["da"][e] = torch.mm(du.t(), x)
            more["db"][e] = torch.mm(dy.t(), s["u"][lo:hi].double()) * ADAPTER_SCALE
    if op == "int8_forward":
        return {"y": out, "a": saved} if case["save"] else {"y": out}
    if op == "int8_dgrad":
        return {"dx": out, "dh1": saved} if saved is not None else {"dx": out}
    return {"y" if op == "adapter_forward" else "dx": out, **more}


if __name__ == "__main__":
    for case in listed() + [draw(random.Random(s)) for s in range(6)]:
        print(case.get("name", "drawn"), case, {k: "%.3g" % v for k, v in work(case).items()})

"""The expert operators in 8-bit floating point, as cases to measure: the ragged
expert product with one scale for each block of 128 (forward and input
gradient, with the activation or its derivative in front), and the gated
feed-forward block made of them (both projections, the activation and the
down projection, forward and backward, with the intermediate kept in 8 bits).

``run`` computes a case with elementary torch operations in 32 bits
(``own = False``) or with the package's entry points (``own = True``);
``exact`` is the definition in 64 bits.

Definitions, for an expert e that owns rows [offsets[e], offsets[e+1]):

  quant(v)       each 128 values of a row (the last block of a row, or of a half of
                 [gate | up], may be shorter) get one power of two 2^c, the least with
                 max|v| <= 448 * 2^c; q = v / 2^c rounded to e4m3, standing for 2^c q
  weights        e4m3 with one power of two for each 128 x 128 block (blocks of W1
                 start anew at its up half)
  fp8_forward    y = quant(v) W_e^T        v = x, or v = A = bf16(act(gate) * up) of x = H1 = [gate | up]
  fp8_dgrad      dx = quant(g) W_e         g = dy, or g = dH1 = bf16(the activation's derivative at H1, times dA = dy)
  glu_forward    H1 = bf16(quant(x) W1_e^T),  A = bf16(act(gate) * up),  y = quant(A) W2_e^T
  glu_dgrad      dA = bf16(quant(dy) W2_e),  dH1 = bf16(...),  dx = quant(dH1) W1_e
"""
import math
import random

import numpy as np
import torch

own = False

SLOPE = {"swiglu": 1.0, "qgeglu": 1.702}
BLOCK = 128          # values that share a scale
TOP = 448.0          # the largest e4m3 value
PAD = 256            # rows of a padded expert block


def _case(name, op, E, rows, routing, K, N, act="none", save=False):
    """Products: x [rows, K], y [rows, N].  Gated blocks: K is the model's width H and N the block's inner width F."""
    return {"name": name, "op": op, "E": E, "rows": rows, "routing": routing, "K": K, "N": N, "act": act, "save": save}


def listed():
    return [
        # one token of a decode step, sent to 8 of 128 experts: latency and the bytes of eight weight matrices
        _case("fp8_token", "fp8_forward", 128, 8, "tokens", 4096, 4096),
        # a small serving batch, about 24 rows for each expert: the gate and up projections of the small-batch workload
        _case("fp8_smallbatch", "fp8_forward", 128, 2880, "uniform", 2688, 3712),
        # a handful of experts with odd sizes: QuickGeGLU in front of the down projection, A kept for an adapter
        _case("fp8_odd_act", "fp8_forward", 5, 777, "uniform", 1048, 2056, act="qgeglu", save=True),
        # the largest workload's gate and up projections, every expert padded to a multiple of 256 rows
        _case("fp8_padded", "fp8_forward", 128, 262144, "padded", 4096, 4096),
        # input gradient of a small batch through the down projection
        _case("fp8_dgrad_smallbatch", "fp8_dgrad", 128, 2880, "uniform", 1856, 2688),
        # input gradient through the gate and up projections with the activation's derivative in front: 32 experts
        _case("fp8_dgrad_act", "fp8_dgrad", 32, 32768, "uniform", 2048, 1536, act="swiglu", save=True),
        # the gated block for one token of a decode step
        _case("glu_token", "glu_forward", 128, 8, "tokens", 4096, 2048, act="swiglu"),
        # the gated block for a small serving batch
        _case("glu_smallbatch", "glu_forward", 128, 2880, "uniform", 2688, 1856, act="swiglu"),
        # a training batch with Zipf-distributed expert sizes, H1 kept for the gradient
        _case("glu_zipf", "glu_forward", 128, 131072, "zipf", 2048, 768, act="swiglu", save=True),
        # a training batch of the largest workload
        _case("glu_padded", "glu_forward", 128, 262144, "padded", 4096, 2048, act="swiglu", save=True),
        # the block's backward pass: the 32-expert workload, and the largest one
        _case("glu_dgrad_uniform", "glu_dgrad", 32, 32768, "uniform", 2048, 768, act="swiglu"),
        _case("glu_dgrad_padded", "glu_dgrad", 128, 262144, "padded", 4096, 2048, act="swiglu"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case with sizes spread over the listed ones' ranges: one row to 131072, widths that
    are any multiples of 8, any number of experts."""
    op = rng.choice(["fp8_forward", "fp8_dgrad", "glu_forward", "glu_forward", "glu_dgrad"])
    rows, E = _spread(rng, 1, 131072), _spread(rng, 1, 128)
    K, N = 8 * _spread(rng, 32, 512), 8 * _spread(rng, 32, 512)
    routing = rng.choice(["uniform", "zipf", "padded" if rows >= PAD else "uniform"])
    if routing == "padded":
        rows = rows // PAD * PAD
    save = False
    if op.startswith("glu"):
        N = max(64, N // 16 * 8)
        act = rng.choice(["swiglu", "swiglu", "qgeglu"])
        save = op == "glu_forward" and rng.random() < 0.5
    else:
        act = rng.choice(["none", "swiglu", "qgeglu"])
        if op == "fp8_dgrad" and act != "none":
            N, save = N // 16 * 16, True
        elif act != "none":
            save = rng.random() < 0.5
    c = _case("", op, E, rows, routing, K, N, act, save)
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


def _blocks(n, halves):
    """(block of each of n rows or columns, number of blocks): blocks of 128 that start anew at each half."""
    each = n // halves
    per = (each + BLOCK - 1) // BLOCK
    at = torch.arange(n, device="cuda")
    return at // each * per + at % each // BLOCK, per * halves


def _weights(E, N, K, halves, gen):
    """Frozen weights in 8 bits with a power of two for each 128 x 128 block: (e4m3 [E, N, K],
    e8m0 [E, blocks of N, blocks of K])."""
    each = N // halves
    nr, nc = (each + BLOCK - 1) // BLOCK, (K + BLOCK - 1) // BLOCK
    q = torch.empty(E, halves, each, K, dtype=torch.float8_e4m3fn, device="cuda")
    s = torch.empty(E, halves, nr, nc, dtype=torch.uint8, device="cuda")
    for e in range(E):
        w = torch.zeros(halves, nr * BLOCK, nc * BLOCK, device="cuda")
        w[:, :each, :K] = torch.randn(halves, each, K, generator=gen, device="cuda").mul_(0.02).to(torch.bfloat16)
        blocks = w.view(halves, nr, BLOCK, nc, BLOCK)
        m, x = torch.frexp(blocks.abs().amax((2, 4)))
        c = x - 9 + (m > TOP / 512).int()
        s[e] = (c + 127).to(torch.uint8)
        unit = torch.ldexp(torch.ones((), device="cuda"), -c)[:, :, None, :, None]
        q[e] = (blocks * unit).view(w.shape)[:, :each, :K].to(torch.float8_e4m3fn)
    q, s = q.view(E, N, K), s.view(E, halves * nr, nc)
    return q, s.view(torch.float8_e8m0fnu)


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

    def rows(width):
        t = torch.empty(M, width, dtype=torch.bfloat16, device="cuda")
        gain = torch.exp(0.5 * torch.randn(width, generator=gen, device="cuda"))     # and so do channels
        for lo in range(0, M, 1 << 14):
            n = min(1 << 14, M - lo)
            t[lo:lo + n] = (torch.randn(n, width, generator=gen, device="cuda") * gain * size[lo:lo + n]).to(torch.bfloat16)
        return t

    s = {"case": case, "offsets": torch.from_numpy(offsets).cuda(),
         "segments": [(e, int(offsets[e]), int(offsets[e + 1])) for e in range(E) if counts[e]]}
    if op == "fp8_forward":
        s["x"] = rows(K if case["act"] == "none" else 2 * K)
        s["w"] = _weights(E, N, K, 1, gen)
    elif op == "fp8_dgrad":
        s["dy"] = rows(N if case["act"] == "none" else N // 2)
        s["h1"] = None if case["act"] == "none" else rows(N)
        s["w"] = _weights(E, N, K, 1 if case["act"] == "none" else 2, gen)
    else:
        if op == "glu_forward":
            s["x"] = rows(K)
        else:
            s["dy"], s["h1"] = rows(K), rows(2 * N)
        s["w1"], s["w2"] = _weights(E, 2 * N, K, 2, gen), _weights(E, K, N, 1, gen)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        # the laid-out frozen weights that a program keeps
        import moe_expert_grouped_ragged_amd as gg
        op = case["op"]
        if op == "fp8_forward":
            s["packed"] = gg.gg_fp8_pack(*s["w"])
        elif op == "fp8_dgrad":
            s["packed"] = gg.gg_fp8_pack_transposed(*s["w"], halves=1 if case["act"] == "none" else 2)
        elif op == "glu_forward":
            s["fc1"], s["fc2"] = gg.gg_fp8_pack(*s["w1"], halves=2), gg.gg_fp8_pack(*s["w2"])
        else:
            s["fc1_t"], s["fc2_t"] = gg.gg_fp8_pack_transposed(*s["w1"], halves=2), gg.gg_fp8_pack_transposed(*s["w2"])
    return s


def _own(s):
    import moe_expert_grouped_ragged_amd as gg
    c = s["case"]
    E, K, N, op = c["E"], c["K"], c["N"], c["op"]
    act = None if c["act"] == "none" else c["act"]
    if op == "fp8_forward":
        y, a = gg.gg_fp8_forward(s["x"], s["offsets"], s["packed"], E, N, K, activation=act, save_a=c["save"])
        return {"y": y, "a": a} if c["save"] else {"y": y}
    if op == "fp8_dgrad":
        dx, dh1 = gg.gg_fp8_dgrad(s["dy"], s["offsets"], s["packed"], E, N, K, halves=2 if act else 1, h1=s["h1"],
                                  activation=act)
        return {"dx": dx, "dh1": dh1} if act else {"dx": dx}
    if op == "glu_forward":
        y, h1 = gg.gg_fp8_glu_forward(s["x"], s["offsets"], s["fc1"], s["fc2"], E, K, N, activation=act, save_h1=c["save"])
        return {"y": y, "h1": h1} if c["save"] else {"y": y}
    return {"dx": gg.gg_fp8_glu_dgrad(s["dy"], s["h1"], s["offsets"], s["fc1_t"], s["fc2_t"], E, K, N, activation=act)}


def _quantized(v, halves=1):
    """What the 8-bit values of float32 rows stand for, as float32."""
    n = v.shape[1]
    each = n // halves
    pad = -each % BLOCK
    b = torch.nn.functional.pad(v.reshape(-1, halves, each), (0, pad)).view(v.shape[0], -1, BLOCK)
    top = b.abs().amax(2, keepdim=True)
    m, x = torch.frexp(top)
    c = torch.where(top > 0, x - 9 + (m > TOP / 512).int(), torch.zeros_like(x))
    q = torch.ldexp(torch.ldexp(b, -c).to(torch.float8_e4m3fn).float(), c)
    return q.view(-1, halves, each + pad)[:, :, :each].reshape(-1, n)


def _dequantized(w, e, halves=1):
    """The matrix that expert e's 8-bit weights stand for, as float32."""
    q, s = w
    scale = torch.ldexp(torch.ones((), device="cuda"), s[e].view(torch.uint8).int() - 127)
    rows, cols = _blocks(q.shape[1], halves)[0], _blocks(q.shape[2], 1)[0]
    return q[e].float() * scale[rows][:, cols]


def _act(h1, k):
    """A = bf16(act(gate) * up)."""
    n = h1.shape[1] // 2
    g, u = h1[:, :n].float(), h1[:, n:].float()
    return (g * torch.sigmoid(k * g) * u).to(torch.bfloat16)


def _act_grad(h1, da, k):
    """dH1 = bf16 of the activation's derivative at H1 times dA."""
    n = h1.shape[1] // 2
    g, u, d = h1[:, :n].float(), h1[:, n:].float(), da.float()
    sg = torch.sigmoid(k * g)
    return torch.cat([d * u * sg * (1 + k * g * (1 - sg)), d * g * sg], 1).to(torch.bfloat16)


def run(s):
    if own:
        return _own(s)
    # A loop over the experts that own rows: their row counts differ, and one product padded
    # to the largest would do many times the work.
    c = s["case"]
    M, K, N, op = c["rows"], c["K"], c["N"], c["op"]
    k = SLOPE.get(c["act"])
    if op == "fp8_forward":
        y = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
        a = _act(s["x"], k) if k else s["x"]
        for e, lo, hi in s["segments"]:
            y[lo:hi] = (_quantized(a[lo:hi].float()) @ _dequantized(s["w"], e).T).to(torch.bfloat16)
        return {"y": y, "a": a} if c["save"] else {"y": y}
    if op == "fp8_dgrad":
        dx = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
        g, halves = (_act_grad(s["h1"], s["dy"], k), 2) if k else (s["dy"], 1)
        for e, lo, hi in s["segments"]:
            dx[lo:hi] = (_quantized(g[lo:hi].float(), halves) @ _dequantized(s["w"], e, halves)).to(torch.bfloat16)
        return {"dx": dx, "dh1": g} if k else {"dx": dx}
    if op == "glu_forward":
        y = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
        h1 = torch.empty(M, 2 * N, dtype=torch.bfloat16, device="cuda")
        for e, lo, hi in s["segments"]:
            h1[lo:hi] = (_quantized(s["x"][lo:hi].float()) @ _dequantized(s["w1"], e, 2).T).to(torch.bfloat16)
            a = _act(h1[lo:hi], k)
            y[lo:hi] = (_quantized(a.float()) @ _dequantized(s["w2"], e).T).to(torch.bfloat16)
        return {"y": y, "h1": h1} if c["save"] else {"y": y}
    dx = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    for e, lo, hi in s["segments"]:
        da = (_quantized(s["dy"][lo:hi].float()) @ _dequantized(s["w2"], e)).to(torch.bfloat16)
        dh1 = _act_grad(s["h1"][lo:hi], da, k)
        dx[lo:hi] = (_quantized(dh1.float(), 2) @ _dequantized(s["w1"], e, 2)).to(torch.bfloat16)
    return {"dx": dx}


def work(case):
    M, K, N = case["rows"], case["K"], case["N"]
    hit = _expected_experts(case)
    act = case["act"] != "none"
    if case["op"] == "fp8_forward":
        read = M * K * (4 if act else 2) + hit * N * K * (1 + 1 / BLOCK ** 2)
        return {"bytes": read + M * N * 2 + (M * K * 2 if case["save"] else 0), "flops": 2.0 * M * N * K}
    if case["op"] == "fp8_dgrad":
        read = M * N * (3 if act else 2) + hit * N * K * (1 + 1 / BLOCK ** 2)
        return {"bytes": read + M * K * 2 + (M * N * 2 if act else 0), "flops": 2.0 * M * N * K}
    weights = 3 * hit * N * K * (1 + 1 / BLOCK ** 2)
    h1 = M * 2 * N * 2 if case["save"] or case["op"] == "glu_dgrad" else 0
    return {"bytes": M * K * 4 + h1 + weights, "flops": 6.0 * M * N * K}


def _levels(v, halves=1):
    """The definition of quant() in 64 bits: the values that v's blocks are rounded to."""
    out = torch.zeros_like(v)
    each = v.shape[1] // halves
    for h in range(halves):
        for lo in range(h * each, (h + 1) * each, BLOCK):
            b = v[:, lo:min(lo + BLOCK, (h + 1) * each)]
            top = torch.amax(torch.abs(b), 1, keepdim=True).clamp_min(2.0 ** -140)
            unit = torch.exp2(torch.ceil(torch.log2(top / 448.0)))
            unit = torch.where(448.0 * unit < top, unit * 2, torch.where(224.0 * unit >= top, unit / 2, unit))
            t = b / unit
            # e4m3: four significant bits, and steps of 2^-9 below 2^-6
            step = torch.exp2(torch.clamp_min(torch.floor(torch.log2(t.abs().clamp_min(2.0 ** -20))), -6.0) - 3.0)
            out[:, lo:lo + b.shape[1]] = torch.round(t / step) * step * unit
    return out


def _matrix(w, e, halves=1):
    """The matrix of expert e in 64 bits, a block at a time."""
    q, s = w[0][e].double(), w[1][e].view(torch.uint8).double() - 127.0
    each = q.shape[0] // halves
    per = s.shape[0] // halves
    for h in range(halves):
        for i in range(per):
            r = slice(h * each + i * BLOCK, min(h * each + (i + 1) * BLOCK, (h + 1) * each))
            q[r] *= torch.exp2(s[h * per + i]).repeat_interleave(BLOCK)[:q.shape[1]]
    return q


def exact(case, seed):
    s = _inputs(case, seed)
    M, K, N, op = case["rows"], case["K"], case["N"], case["op"]
    k = SLOPE.get(case["act"], 0.0)

    def empty(width):
        return torch.empty(M, width, dtype=torch.float64, device="cuda")

    def bf16(t):
        return t.to(torch.bfloat16).double()

    def activated(h):
        gate, up = torch.chunk(h, 2, 1)
        return gate / (1.0 + torch.exp(-k * gate)) * up

    def derived(h, d):
        gate, up = torch.chunk(h, 2, 1)
        z = torch.exp(-k * gate)
        return torch.cat([d * up * (1.0 + z + k * gate * z) / (1.0 + z) ** 2, d * gate / (1.0 + z)], 1)

    # H1, A, dA and dH1 are rounded to bf16 where they are defined, before they are used or quantized.
    out, more = empty(N if op == "fp8_forward" else K), {}
    if op == "fp8_forward" and case["save"]:
        more["a"] = empty(K)
    if op == "fp8_dgrad" and k:
        more["dh1"] = empty(N)
    if op == "glu_forward" and case["save"]:
        more["h1"] = empty(2 * N)
    for e, lo, hi in s["segments"]:
        if op == "fp8_forward":
            v = s["x"][lo:hi].double()
            if k:
                a = activated(v)
                if case["save"]:
                    more["a"][lo:hi] = a
                v = bf16(a)
            out[lo:hi] = torch.mm(_levels(v), _matrix(s["w"], e).t().contiguous())
        elif op == "fp8_dgrad":
            v = s["dy"][lo:hi].double()
            if k:
                more["dh1"][lo:hi] = derived(s["h1"][lo:hi].double(), v)
                v = bf16(more["dh1"][lo:hi])
            halves = 2 if k else 1
            out[lo:hi] = torch.mm(_levels(v, halves), _matrix(s["w"], e, halves))
        elif op == "glu_forward":
            h = torch.mm(_levels(s["x"][lo:hi].double()), _matrix(s["w1"], e, 2).t().contiguous())
            if case["save"]:
                more["h1"][lo:hi] = h
            a = bf16(activated(bf16(h)))
            out[lo:hi] = torch.mm(_levels(a), _matrix(s["w2"], e).t().contiguous())
        else:
            da = bf16(torch.mm(_levels(s["dy"][lo:hi].double()), _matrix(s["w2"], e)))
            dh = bf16(derived(s["h1"][lo:hi].double(), da))
            out[lo:hi] = torch.mm(_levels(dh, 2), _matrix(s["w1"], e, 2))
    return {"y" if op in ("fp8_forward", "glu_forward") else "dx": out, **more}


if __name__ == "__main__":
    for case in listed() + [draw(random.Random(s)) for s in range(6)]:
        print(case.get("name", "drawn"), case, {k: "%.3g" % v for k, v in work(case).items()})

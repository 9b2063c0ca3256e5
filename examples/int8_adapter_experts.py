"""Low-rank adapters trained next to a frozen 8-bit expert layer, then one token served.

A teacher layer with other weights gives the targets; the adapters of the
8-bit layer learn the difference with plain SGD on fp32 copies.

    python examples/int8_adapter_experts.py [--steps N]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import moe_expert_grouped_ragged_amd as gg   # noqa: E402
import workload                              # noqa: E402


def main(steps: int = 40, seed: int = 7):
    """Returns (losses of the steps, the served token's output, the same row of a training batch's)."""
    E, H, F, r, scale, dev = 8, 256, 384, 8, 2.0, torch.device("cuda:0")
    counts = [120, 0, 33, 256, 7, 64, 300, 1]                  # ragged, one expert without tokens
    case = workload.custom_case(counts, H, F, seed=seed)
    x, offsets = case.x.to(dev), torch.from_numpy(case.offsets).to(dev)
    experts = gg.int8_experts(case.w1.to(dev), case.w2.to(dev))

    gen = torch.Generator().manual_seed(seed)
    shapes = [(E, r, H), (E, 2 * F, r), (E, r, F), (E, H, r)]      # a1, b1, a2, b2
    teacher = [(torch.randn(s, generator=gen) * 0.05).to(torch.bfloat16).to(dev) for s in shapes]
    target = gg.Int8AdapterExpertMLP.apply(x, offsets, experts, *teacher, scale)
    # a starts random and b at zero, so the first output is the frozen layer's
    master = [(torch.randn(s, generator=gen) * 0.05).to(dev) if i % 2 == 0 else torch.zeros(s, device=dev)
              for i, s in enumerate(shapes)]
    losses, lr = [], 4.0
    for _ in range(steps):
        params = [m.to(torch.bfloat16).requires_grad_(True) for m in master]
        y = gg.Int8AdapterExpertMLP.apply(x, offsets, experts, *params, scale)
        loss = (y.float() - target.float()).square().sum() / x.shape[0]
        loss.backward()
        for m, p in zip(master, params):
            m -= lr * p.grad.float()
        losses.append(float(loss.detach()))

    # serving: one token, routed to expert 3, as a batch of its own
    params = [m.to(torch.bfloat16) for m in master]
    batch = gg.Int8AdapterExpertMLP.apply(x, offsets, experts, *params, scale)
    row = int(case.offsets[3]) + 5
    one = torch.zeros(E + 1, dtype=torch.int64, device=dev)
    one[4:] = 1
    token = gg.Int8AdapterExpertMLP.apply(x[row:row + 1].contiguous(), one, experts, *params, scale)
    return losses, token[0], batch[row]


if __name__ == "__main__":
    ap = argparse.ArgumentParser(description=__doc__)
    ap.add_argument("--steps", type=int, default=40)
    losses, token, batch = main(ap.parse_args().steps)
    print("loss %.4f -> %.4f" % (losses[0], losses[-1]))
    print("one token alone against its row in the batch: largest difference %.3g of %.3g" %
          (float((token.float() - batch.float()).abs().max()), float(batch.float().abs().max())))

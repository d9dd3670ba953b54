"""Trains a two-layer network on a synthetic regression with the linear-layer
operators together: the layers' products and gradients in 8 bits (fp8_linear),
the weights' updates orthogonalised (newton_schulz), and the trained weights
quantised once and served with linear_fp8, a prompt and single rows.

    python examples/train_linear_fp8.py [--steps 60] [--tokens 2048] [--width 1024]
"""
import argparse
import math
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


def train(steps=60, tokens=2048, width=1024, hidden=1536, lr=0.05, momentum=0.9, seed=0):
    """(losses by step, final weights, a batch of inputs and its targets)."""
    import torch

    import thread_block_smem_gb300 as swz
    g = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")
    # what is to be learnt: a random layer of the same form
    target = [randn(hidden, width) / math.sqrt(width), randn(width, hidden) / math.sqrt(hidden)]
    # fp32 weights, rounded to bf16 where the layers read them
    weights = [0.5 * randn(hidden, width) / math.sqrt(width),
               0.5 * randn(width, hidden) / math.sqrt(hidden)]
    moments = [torch.zeros_like(w) for w in weights]
    losses = []
    for step in range(steps):
        x = randn(tokens, width).bfloat16()
        want = torch.relu(x.float() @ target[0].t()) @ target[1].t()
        params = [w.bfloat16().requires_grad_() for w in weights]
        y = swz.fp8_linear(torch.relu(swz.fp8_linear(x, params[0])), params[1])
        loss = (y.float() - want).square().mean()
        loss.backward()
        for w, m, p in zip(weights, moments, params):
            m.mul_(momentum).add_(p.grad.float())
            # singular values near 1: a step of lr per direction, scaled by the shape
            update = swz.newton_schulz(m)
            w.sub_(lr * (1 - step / steps) * math.sqrt(max(1.0, w.shape[0] / w.shape[1])) *
                   update.float())
        losses.append(loss.detach())
    swz.check_status()
    return [float(v) for v in losses], weights, x, want


def serve(weights, x):
    """The network on x from weights quantised once: (q, scales) of each layer."""
    import torch

    import thread_block_smem_gb300 as swz
    kept = [swz.quantize_fp8(w.bfloat16(), "square") for w in weights]
    return swz.linear_fp8(torch.relu(swz.linear_fp8(x, *kept[0])), *kept[1])


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawTextHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--width", type=int, default=1024)
    a = ap.parse_args()
    losses, weights, x, want = train(a.steps, a.tokens, a.width)
    print("loss %.4f -> %.4f in %d steps" % (losses[0], losses[-1], len(losses)))
    y = serve(weights, x)
    one = serve(weights, x[:1])
    print("served: mean square error %.4f; one row apart from the batch: %s" % (
        (y.float() - want).square().mean(), "same" if bool((one == y[:1]).all()) else
        "largest difference %.3g" % (one.float() - y[:1].float()).abs().max()))


if __name__ == "__main__":
    main()

"""Trains a pre-norm residual block on a synthetic regression and serves it:

    y = x + W2 silu(W1 layer_norm(x))

in training with the products in 8-bit floating point (fp8_linear), the layer norm
and its gradient (layer_norm), the gradients clipped together into 32-bit buffers
(clip_grad_norm) and the weights' updates orthogonalised (newton_schulz); then with
weights kept in 8-bit integers, a scale for each output channel (quantize_int8,
linear_int8), a prompt and single tokens.

    python examples/train_block.py [--steps 60] [--tokens 2048] [--width 1024]
"""
import argparse
import math
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))


def block(x, params):
    """y of x (tokens x width, bf16); params: norm weight and bias, W1, W2."""
    import torch

    import thread_block_smem_gb300 as swz
    g, b, w1, w2 = params
    h = swz.fp8_linear(swz.layer_norm(x, g, b), w1)
    return x + swz.fp8_linear(torch.nn.functional.silu(h), w2)


def start(width, hidden, g):
    """Norm weight and bias, W1, W2 in fp32."""
    import torch
    return [torch.ones(width, device="cuda"), torch.zeros(width, device="cuda"),
            torch.randn((hidden, width), generator=g, device="cuda") / math.sqrt(width),
            0.5 * torch.randn((width, hidden), generator=g, device="cuda") / math.sqrt(hidden)]


def train(steps=60, tokens=2048, width=1024, hidden=1536, lr=0.05, momentum=0.9, max_norm=1.0, seed=0):
    """(losses and gradient norms by step, final weights, a batch of inputs)."""
    import torch

    import thread_block_smem_gb300 as swz
    g = torch.Generator(device="cuda").manual_seed(seed)
    target = start(width, hidden, g)
    weights = start(width, hidden, g)
    moments = [torch.zeros_like(w) for w in weights]
    clipped = [torch.empty_like(w) for w in weights]
    log = []
    for step in range(steps):
        x = torch.randn((tokens, width), generator=g, device="cuda").bfloat16()
        n = torch.nn.functional.layer_norm(x.float(), (width,), target[0], target[1])
        want = x.float() + torch.nn.functional.silu(n @ target[2].t()) @ target[3].t()
        # bf16 weights for the products, fp32 for the norm
        params = [w.clone() if w.dim() == 1 else w.bfloat16() for w in weights]
        for p in params:
            p.requires_grad_()
        loss = (block(x, params).float() - want).square().mean()
        loss.backward()
        norm = swz.clip_grad_norm([p.grad for p in params], max_norm, out=clipped)
        scale = lr * (1 - step / steps)
        for w, m, c in zip(weights, moments, clipped):
            m.mul_(momentum).add_(c)
            if w.dim() == 1:
                w.sub_(scale * m)
            else:
                w.sub_(scale * math.sqrt(max(1.0, w.shape[0] / w.shape[1])) * swz.newton_schulz(m).float())
        log.append((loss.detach(), norm))
    swz.check_status()
    return [(float(a), float(b)) for a, b in log], weights, x


def keep(weights):
    """What serving keeps: the norm's weight and bias, W1 and W2 as 8-bit integers."""
    import thread_block_smem_gb300 as swz
    return [weights[0], weights[1], swz.quantize_int8(weights[2]), swz.quantize_int8(weights[3])]


def serve(kept, x):
    """The block on x (tokens x width, bf16)."""
    import torch

    import thread_block_smem_gb300 as swz
    n, _, _ = swz.layer_norm_forward(x, kept[0], kept[1])
    h = torch.nn.functional.silu(swz.linear_int8(n, *kept[2]))
    return x + swz.linear_int8(h, *kept[3])


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawTextHelpFormatter)
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--tokens", type=int, default=2048)
    ap.add_argument("--width", type=int, default=1024)
    a = ap.parse_args()
    log, weights, x = train(a.steps, a.tokens, a.width)
    print("loss %.4f -> %.4f, gradient norm %.3f -> %.3f in %d steps" % (
        log[0][0], log[-1][0], log[0][1], log[-1][1], len(log)))
    kept = keep(weights)
    y, one = serve(kept, x), serve(kept, x[:1])
    with_8_bit_floats = block(x, [w if w.dim() == 1 else w.bfloat16() for w in weights])
    print("served: %.4f of the block's part off what training computes; one token apart from the "
          "batch: largest difference %.3g" % (
              (y.float() - with_8_bit_floats.float()).norm() / (with_8_bit_floats.float() - x.float()).norm(),
              (one.float() - y[:1].float()).abs().max()))


if __name__ == "__main__":
    main()

"""An expert layer trained with the grouped products, then served with int8 weights.

Every token goes to one of `groups` experts, each relu(x W1) W2.  A step sorts
the tokens by expert, runs both grouped products forward, their gradients of the
rows back (the same weights, read the other way round), and adds the gradients
of the weights of two micro-batches up in fp32.  The target is another layer of
the same shape, so the loss falls.  Afterwards a projection of the layer's result
is served with int8 weights, quantized once, for one token and for many.

    python examples/expert_layer.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import tiled_tensor_core_02_gb300 as ttc  # noqa: E402


def route(router, x, groups):
    """Token order by expert and the experts' offsets, all on the device."""
    expert = (x.float() @ router).argmax(dim=1)
    counts = torch.bincount(expert, minlength=groups)
    offsets = torch.zeros(groups + 1, dtype=torch.int32, device=x.device)
    offsets[1:] = counts.cumsum(0)
    return expert.argsort(stable=True), offsets


def forward(x, offsets, w1, w2):
    h = ttc.gemm_grouped(x, w1, offsets, act="relu")
    return h, ttc.gemm_grouped(h, w2, offsets)


def train(tokens=2048, groups=4, width=128, hidden=256, steps=60, rate=0.03, seed=0):
    """Mean squared errors, one a step, and the trained layer (router, w1, w2)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *shape: torch.randn(shape, generator=gen, device="cuda")
    router = normal(width, groups)
    layer = lambda: [normal(groups, width, hidden) / width ** 0.5, normal(groups, hidden, width) / hidden ** 0.5]
    target = [w.bfloat16() for w in layer()]
    master = layer()
    grads = [torch.empty_like(w) for w in master]
    losses = []
    for _ in range(steps):
        w1, w2 = (w.bfloat16() for w in master)
        loss = 0.0
        for part in range(2):
            x = normal(tokens // 2, width).bfloat16()
            order, offsets = route(router, x, groups)
            x = x[order]
            want = forward(x, offsets, *target)[1].float()
            h, y = forward(x, offsets, w1, w2)
            diff = y.float() - want
            loss = loss + diff.square().mean() / 2
            dy = (diff * (groups / tokens)).bfloat16()  # an expert's mean over its tokens
            dh = ttc.gemm_grouped(dy, w2.transpose(1, 2), offsets)
            dh = torch.where(h > 0, dh, torch.zeros_like(dh))
            beta = float(part)  # the first micro-batch sets the gradients, the second adds
            ttc.gemm_grouped_wgrad(h, dy, offsets, c=grads[1], out=grads[1], beta=beta)
            ttc.gemm_grouped_wgrad(x, dh, offsets, c=grads[0], out=grads[0], beta=beta)
        for w, g in zip(master, grads):
            w.sub_(g, alpha=rate)
        losses.append(loss)
    return [float(v) for v in losses], (router, *(w.bfloat16() for w in master))


def serve(layer, outputs=4096, counts=(1, 24, 512), seed=1):
    """Relative error of an int8 projection of the layer's result, by number of tokens."""
    router, w1, w2 = layer
    groups, width = w1.shape[:2]
    gen = torch.Generator(device="cuda").manual_seed(seed)
    projection = torch.randn((outputs, width), generator=gen, device="cuda") / width ** 0.5
    q, q_scale = ttc.quantize_rows(projection)  # once, when the model is loaded
    errors = {}
    for tokens in counts:
        x = torch.randn((tokens, width), generator=gen, device="cuda").bfloat16()
        order, offsets = route(router, x, groups)
        y = forward(x[order], offsets, w1, w2)[1]
        rows, scale = ttc.quantize_rows(y)
        logits = ttc.gemm_i8_scaled(rows, scale, q, q_scale, out_dtype=torch.float32)
        exact = y.double() @ projection.double().T
        errors[tokens] = float((logits.double() - exact).norm() / exact.norm())
    return errors


def main():
    losses, layer = train()
    print("mean squared error:", " ".join(f"{v:.4f}" for v in losses[::12] + losses[-1:]))
    for tokens, e in serve(layer).items():
        print(f"int8 projection of {tokens} tokens: relative error {e:.4f}")


if __name__ == "__main__":
    main()

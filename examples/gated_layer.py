"""A gated feed-forward layer trained with the gated block, then served in 8-bit floats.

The layer is silu(x Wg) * (x Wu) Wd; both first weights are one matrix, gate on top of the
other.  A step keeps the two projections, reads them in the gradient (which also gives the
product again for Wd's gradient), and adds the gradients of two micro-batches up in
fp32.  The target is another layer of the same shape.  Afterwards the weights are quantized
once, in blocks of 128 x 128, and the layer runs on them for one token and for many.

    python examples/gated_layer.py
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import tiled_tensor_core_02_gb300 as ttc  # noqa: E402


def forward(x, w, wd, keep=False):
    """The layer's result, with keep what backward needs too."""
    n = wd.shape[1]
    gate, up = w[:n].t(), w[n:].t()
    if not keep:
        return ttc.gemm(ttc.gemm_gated(x, gate, up), wd.t())
    h, pre = ttc.gemm_gated(x, gate, up, pre=True)
    return ttc.gemm(h, wd.t()), pre


def backward(x, w, wd, pre, dy, dw, dwd, add):
    """The gradient of x; those of the weights go into dw and dwd (fp32), or are added to them."""
    h = torch.empty((x.shape[0], wd.shape[1]), dtype=x.dtype, device=x.device)
    dpre = ttc.gemm_gated_grad(dy, wd, pre, pre, out=h)  # in the kept projections' place
    rows = torch.tensor([0, x.shape[0]], dtype=torch.int32, device=x.device)
    beta = 1.0 if add else 0.0
    ttc.gemm_grouped_wgrad(dpre, x, rows, c=dw[None], out=dw[None], beta=beta)
    ttc.gemm_grouped_wgrad(dy, h, rows, c=dwd[None], out=dwd[None], beta=beta)
    return ttc.gemm(dpre, w)


def make(gen, width, hidden):
    normal = lambda *shape: torch.randn(shape, generator=gen, device="cuda")
    return [normal(2 * hidden, width) / width ** 0.5, normal(width, hidden) / hidden ** 0.5]


def train(tokens=1024, width=128, hidden=384, steps=60, rate=0.3, seed=0):
    """Mean squared errors, one a step, and the trained weights."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    target = [w.bfloat16() for w in make(gen, width, hidden)]
    master = make(gen, width, hidden)
    grads = [torch.empty_like(w) for w in master]
    losses = []
    for _ in range(steps):
        weights = [w.bfloat16() for w in master]
        loss = 0.0
        for part in range(2):
            x = torch.randn((tokens // 2, width), generator=gen, device="cuda").bfloat16()
            y, pre = forward(x, *weights, keep=True)
            diff = y.float() - forward(x, *target).float()
            loss = loss + diff.square().mean() / 2
            backward(x, *weights, pre, (diff / (tokens * width) * 64).bfloat16(), *grads, add=part > 0)
        for w, g in zip(master, grads):
            w.sub_(g, alpha=rate / 64 * width)
        losses.append(loss)
    return [float(v) for v in losses], [w.bfloat16() for w in master]


def serve(weights, counts=(1, 24, 512), seed=1):
    """Relative error of the layer on 8-bit weights and tokens, by number of tokens."""
    w, wd = weights
    n = wd.shape[1]
    quantized = [ttc.quantize_blocks(v, block_rows=128) for v in (w, wd)]  # once, when the model is loaded
    gen = torch.Generator(device="cuda").manual_seed(seed)
    errors = {}
    for tokens in counts:
        x = torch.randn((tokens, w.shape[1]), generator=gen, device="cuda").bfloat16()
        pre = ttc.gemm_f8_blocks(*ttc.quantize_blocks(x), *quantized[0])
        h = torch.nn.functional.silu(pre[:, :n].float()) * pre[:, n:].float()
        y = ttc.gemm_f8_blocks(*ttc.quantize_blocks(h), *quantized[1], out_dtype=torch.float32)
        pre = x.double() @ w.double().t()
        exact = (torch.nn.functional.silu(pre[:, :n]) * pre[:, n:]) @ wd.double().t()
        errors[tokens] = float((y.double() - exact).norm() / exact.norm())
    return errors


def main():
    losses, weights = train()
    print("mean squared error:", " ".join(f"{v:.4f}" for v in losses[::12] + losses[-1:]))
    for tokens, e in serve(weights).items():
        print(f"8-bit layer, {tokens} tokens: relative error {e:.4f}")


if __name__ == "__main__":
    main()

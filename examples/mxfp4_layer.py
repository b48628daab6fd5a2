"""A routed SwiGLU layer in 4 bits, from fine-tuning to serving, on one GPU.

    python examples/mxfp4_layer.py

1. One fine-tuning step: the three products of the layer are differentiable MXFP4 products (forward in 4 bits,
   gradients in 8), over tokens grouped by expert.
2. The weights are quantized once for serving.
3. A prompt's tokens go through the grouped products, with SwiGLU and the quantization of h in one kernel.
4. The tokens that follow go through ``MxMoeTokens``, a few at a time, over the same weights.

Random weights and tokens; prints how far the two serving paths are apart and what each takes."""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mxfp8_precision_moe_gb300 as mx  # noqa: E402


def dispatch(logits: torch.Tensor, top_k: int, multiple: int = 1):
    """Tokens grouped by expert: for each of M rows the token it takes (-1: padding, to make every group a
    multiple of ``multiple`` rows) and its weight, and the groups' end rows."""
    T, E = logits.shape
    top, experts = logits.topk(top_k, dim=1)
    weights = top.softmax(1).flatten()
    experts = experts.flatten()
    order = experts.argsort(stable=True)
    counts = torch.bincount(experts, minlength=E)
    padded = (counts + multiple - 1) // multiple * multiple
    ends, starts = padded.cumsum(0), counts.cumsum(0) - counts
    place = torch.arange(T * top_k, device=logits.device) - starts[experts[order]] + (ends - padded)[experts[order]]
    token = torch.full((int(ends[-1]),), -1, dtype=torch.long, device=logits.device)
    weight = torch.zeros(token.shape, device=logits.device)
    token[place] = order // top_k
    weight[place] = weights[order]
    return token, weight, ends.to(torch.int32)


def gather(x: torch.Tensor, token: torch.Tensor) -> torch.Tensor:
    return torch.where((token >= 0)[:, None], x[token.clamp_min(0)], 0)


def combine(y: torch.Tensor, token: torch.Tensor, weight: torch.Tensor, T: int) -> torch.Tensor:
    out = torch.zeros((T, y.shape[1]), device=y.device)
    return out.index_add(0, token.clamp_min(0), y.float() * weight[:, None])


def train_layer(x, logits, gate, up, down, top_k: int) -> torch.Tensor:
    """The layer for training: y [T, D], differentiable in x and the weights."""
    token, weight, offs = dispatch(logits, top_k, multiple=32)
    rows = gather(x, token)
    h1 = mx.to_mxfp4_then_scaled_grouped_mm(rows, gate, offs)
    h3 = mx.to_mxfp4_then_scaled_grouped_mm(rows, up, offs, check_offsets=False)
    h = torch.nn.functional.silu(h1.float()) * h3.float()
    y = mx.to_mxfp4_then_scaled_grouped_mm(h.bfloat16(), down, offs, check_offsets=False)
    return combine(y, token, weight, x.shape[0])


class ServingLayer:
    """The layer for serving: one set of MXFP4 weights, a path for prompts and one for the tokens that follow."""

    def __init__(self, gate, up, down, top_k: int):
        self.top_k = top_k
        self.gate, self.up, self.down = (mx.mxfp4_quantize_3d_experts(w) for w in (gate, up, down))
        self.step = mx.MxMoeTokens(self.gate, self.up, self.down, top_k)

    @torch.no_grad()
    def prompt(self, x: torch.Tensor, logits: torch.Tensor) -> torch.Tensor:
        token, weight, offs = dispatch(logits, self.top_k)
        q = mx.mxfp4_quantize_2d(x[token], offs=offs)
        h1 = mx.mxfp4_grouped_mm_fwd(*q, *self.gate, offs)
        h3 = mx.mxfp4_grouped_mm_fwd(*q, *self.up, offs)
        y = mx.mxfp4_grouped_mm_fwd(*mx.mxfp4_swiglu_quantize(h1, h3, offs=offs), *self.down, offs)
        return combine(y, token, weight, x.shape[0]).bfloat16()

    @torch.no_grad()
    def tokens(self, x: torch.Tensor, logits: torch.Tensor) -> torch.Tensor:
        return self.step(x, logits)


def run(E: int = 8, D: int = 1024, H: int = 2048, top_k: int = 2, prompt: int = 500, follow: int = 4, seed: int = 0):
    """-> (weight gradients, prompt outputs of the last ``follow`` tokens, the same tokens' outputs by themselves)."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*shape, scale=1.0):
        return (torch.randn(*shape, device="cuda", generator=g) * scale).bfloat16()

    gate, up, down = rand(E, H, D, scale=D ** -0.5), rand(E, H, D, scale=D ** -0.5), rand(E, D, H, scale=H ** -0.5)
    x, logits = rand(prompt, D), rand(prompt, E).float()
    leaves = [w.requires_grad_(True) for w in (gate, up, down)]
    loss = (train_layer(x, logits, *leaves, top_k) - x.float()).square().mean()
    grads = torch.autograd.grad(loss, leaves)
    with torch.no_grad():
        for w, d in zip(leaves, grads):
            w -= 0.1 * d
    layer = ServingLayer(*(w.detach() for w in leaves), top_k)
    return grads, layer.prompt(x, logits)[-follow:], layer.tokens(x[-follow:], logits[-follow:]), layer, (x, logits)


def main() -> None:
    def time(f, n=50):
        f()
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(n):
            f()
        b.record()
        b.synchronize()
        return a.elapsed_time(b) * 1e3 / n

    grads, many, few, layer, (x, logits) = run()
    print("gradient norms", [round(float(d.float().norm()), 4) for d in grads])
    apart = (many.float() - few.float()).norm() / few.float().norm()
    print(f"the same tokens in the prompt and by themselves: {float(apart):.4f} apart (relative)")
    print(f"prompt of {x.shape[0]} tokens {time(lambda: layer.prompt(x, logits)):.0f} us, "
          f"4 tokens {time(lambda: layer.tokens(x[-4:], logits[-4:])):.1f} us")


if __name__ == "__main__":
    main()

"""A gated feed-forward layer in 8 bits: training and serving.

    python examples/fp8_mlp.py [--tokens 512] [--width 512] [--hidden 1376] [--steps 20]

y = (silu(x Wg^T) * (x Wu^T)) Wd^T. Master weights are fp32; every step
quantises them to 128 x 128 blocks in both directions (iris_fp8_quantize), runs
the products in 8 bits (iris_fp8_mm) with the gated activation between them
(iris_fp8_swiglu), and keeps three 8-bit matrices for the backward pass: x, gate
and up. The backward pass (iris_fp8_swiglu_bwd) recomputes h from them; weight
gradients come out in fp32. The example fits a random target layer, prints the
loss, and then runs one token through the layer as a decoding step would.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gemm_collective_tile_amd as il  # noqa: E402


class Weight8:
    """A weight (out, in) in 8 bits: `fwd` for x W^T, `bwd` (in, out) for dy W."""

    def __init__(self, out_features, in_features):
        self.version = 0
        self.fwd = il.iris_fp8_empty(out_features, in_features, block=128)
        self.bwd = il.iris_fp8_empty(in_features, out_features, block=128)

    def set(self, w):
        il.iris_fp8_quantize(w, self.fwd, self.bwd)
        self.version += 1


class FeedForward(torch.autograd.Function):
    """x (tokens, width) 16-bit; wg, wu (hidden, width), wd (width, hidden) fp32;
    g8, u8, d8 their Weight8."""

    @staticmethod
    def forward(ctx, x, wg, wu, wd, g8, u8, d8):
        n, width = x.shape
        hidden = wg.shape[0]
        x8 = il.iris_fp8_empty(n, width)
        il.iris_fp8_quantize(x, x8)
        gate, up = (torch.empty((n, hidden), dtype=x.dtype, device=x.device) for _ in range(2))
        il.iris_fp8_mm(gate, x8, g8.fwd)
        il.iris_fp8_mm(up, x8, u8.fwd)
        h8 = il.iris_fp8_empty(n, hidden)
        keep = any(ctx.needs_input_grad)
        gate8, up8 = (il.iris_fp8_empty(n, hidden) if keep else None for _ in range(2))
        il.iris_fp8_swiglu(h8, gate, up, gate8, up8)
        y = torch.empty((n, wd.shape[0]), dtype=x.dtype, device=x.device)
        il.iris_fp8_mm(y, h8, d8.fwd)
        ctx.kept, ctx.weights = (x8, gate8, up8), (g8, u8, d8)
        ctx.versions = [w.version for w in ctx.weights]
        return y

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy):
        (x8, gate8, up8), (g8, u8, d8) = ctx.kept, ctx.weights
        if [w.version for w in ctx.weights] != ctx.versions:
            raise RuntimeError("the 8-bit weights have been set anew since the forward pass")
        for_x, for_wg, for_wu, for_wd = ctx.needs_input_grad[:4]
        n, width = x8.shape
        hidden = gate8.shape[1]
        dy = dy.contiguous()
        dy8, dy8_t = il.iris_fp8_empty(n, width), il.iris_fp8_empty(width, n) if for_wd else None
        il.iris_fp8_quantize(dy, dy8, dy8_t)
        dh = torch.empty((n, hidden), dtype=dy.dtype, device=dy.device)
        il.iris_fp8_mm(dh, dy8, d8.bwd)
        dg, du = il.iris_fp8_empty(n, hidden), il.iris_fp8_empty(n, hidden)
        dg_t, du_t, h_t = (il.iris_fp8_empty(hidden, n) if wanted else None for wanted in (for_wg, for_wu, for_wd))
        il.iris_fp8_swiglu_bwd(dg, du, dh, gate8, up8, dg_t, du_t, h_t)
        dx = dwg = dwu = dwd = None
        if for_x:
            dx = torch.empty((n, width), dtype=torch.float32, device=dy.device)
            il.iris_fp8_mm(dx, dg, g8.bwd)
            il.iris_fp8_mm(dx, du, u8.bwd, accumulate=True)
            dx = dx.to(dy.dtype)
        if for_wg or for_wu:
            x8_t = il.iris_fp8_empty(width, n)
            il.iris_fp8_quantize(x8, None, x8_t)
        if for_wg:
            dwg = torch.empty((hidden, width), dtype=torch.float32, device=dy.device)
            il.iris_fp8_mm(dwg, dg_t, x8_t)
        if for_wu:
            dwu = torch.empty((hidden, width), dtype=torch.float32, device=dy.device)
            il.iris_fp8_mm(dwu, du_t, x8_t)
        if for_wd:
            dwd = torch.empty((width, hidden), dtype=torch.float32, device=dy.device)
            il.iris_fp8_mm(dwd, dy8_t, h_t)
        return dx, dwg, dwu, dwd, None, None, None


class Layer(torch.nn.Module):
    def __init__(self, width, hidden, device="cuda"):
        super().__init__()
        self.wg = torch.nn.Parameter(torch.randn(hidden, width, device=device) / width ** 0.5)
        self.wu = torch.nn.Parameter(torch.randn(hidden, width, device=device) / width ** 0.5)
        self.wd = torch.nn.Parameter(torch.randn(width, hidden, device=device) / hidden ** 0.5)
        self.w8 = Weight8(hidden, width), Weight8(hidden, width), Weight8(width, hidden)
        self.refresh()

    @torch.no_grad()
    def refresh(self):
        """After the weights have changed: their 8-bit copies."""
        for w8, w in zip(self.w8, (self.wg, self.wu, self.wd)):
            w8.set(w)

    def forward(self, x):
        return FeedForward.apply(x, self.wg, self.wu, self.wd, *self.w8)


def train(tokens, width, hidden, steps, lr=0.02, seed=0):
    """Losses of `steps` gradient steps towards a random layer's outputs."""
    torch.manual_seed(seed)
    layer, goal = Layer(width, hidden), Layer(width, hidden)
    losses = []
    for _ in range(steps):
        x = torch.randn(tokens, width, device="cuda").to(torch.bfloat16)
        with torch.no_grad():
            target = goal(x).float()
        loss = (layer(x).float() - target).square().mean()
        loss.backward()
        with torch.no_grad():
            for w in layer.parameters():
                w -= lr * w.norm() / (w.grad.norm() + 1e-12) * w.grad   # a step of lr of the weight's own size
                w.grad = None
        layer.refresh()
        losses.append(loss.detach())
    return layer, [float(v) for v in losses]


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--width", type=int, default=512)
    ap.add_argument("--hidden", type=int, default=1376)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    layer, losses = train(a.tokens, a.width, a.hidden, a.steps)
    print("loss: " + " ".join(f"{v:.4f}" for v in losses))
    with torch.no_grad():
        y = layer(torch.randn(1, a.width, device="cuda").to(torch.bfloat16))
    print(f"one token: output norm {float(y.float().norm()):.3f}")


if __name__ == "__main__":
    main()

"""A residual feed-forward block in 8 bits around an ungated layer: training and serving.

    python examples/fp8_block.py [--tokens 512] [--width 512] [--hidden 1376] [--steps 20]

    n = norm(x) pre_w,  h = gelu(n W1^T + b1),  y = h W2^T + b2
    r = x + alpha gate m norm(y) post_w

x and r are the 32-bit residual stream, m a dropout mask that is computed and never
stored. The norm (iris_block_norm) writes n in 8 bits for the first product, whose
epilogue (iris_fp8_mm_act) adds the bias, keeps z and writes h in 8 bits for the
second; the second norm, the gate, the dropout and the residual sum are one call. The
backward pass goes through the same operators (iris_block_norm_bwd,
iris_fp8_mm_act_bwd) and the quantiser that turns 8-bit matrices around for the weight
gradients. Serving makes the same calls for one token, without dropout and without what
the backward pass needs.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import gemm_collective_tile_amd as il  # noqa: E402
from fp8_mlp import Weight8  # noqa: E402

NAMES = ("w1", "b1", "w2", "b2", "pre_w", "post_w", "gate")


def forward(block, x, dropout, keep):
    """r, and what the backward pass needs."""
    n, width = x.shape
    hidden = block.w1.shape[0]
    half, dev = torch.bfloat16, x.device
    before = il.BlockNorm(pre_w=block.pre_w.detach())
    after = il.BlockNorm(post=True, post_w=block.post_w.detach(), gate=block.gate.detach(), alpha=block.alpha, dropout=dropout)
    n8, h8 = il.iris_fp8_empty(n, width, device=dev), il.iris_fp8_empty(n, hidden, device=dev)
    stats = [torch.empty((n, 4), device=dev) if keep else None for _ in range(2)]
    z = torch.empty((n, hidden), dtype=half, device=dev) if keep else None
    y, r = torch.empty((n, width), dtype=half, device=dev), torch.empty_like(x)
    il.iris_block_norm(x, before, q=n8, stats=stats[0])
    il.iris_fp8_mm_act(None, n8, block.w1_8.fwd, act="gelu", bias=block.b1.detach().to(half), z=z, q=h8, dtype=half)
    il.iris_fp8_mm_act(y, h8, block.w2_8.fwd, bias=block.b2.detach().to(half))
    il.iris_block_norm(x, after, y=y, r=r, stats=stats[1])
    return r, (y, z, n8, h8, stats, before, after)


class BlockFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, block, dropout, x, *params):
        keep = any(ctx.needs_input_grad)
        if keep and dropout is not None:
            # the backward pass takes this pass's mask, wherever the caller's handle and counter have moved by then
            at = dropout.counter
            dropout = il.Dropout(dropout.p, dropout.seed, dropout.offset, None if at is None else at.clone())
        r, kept = forward(block, x, dropout, keep)
        if keep:
            # what the backward pass reads of the caller's: autograd refuses it if it has changed by then
            ctx.save_for_backward(x, block.pre_w, block.post_w, block.gate)
            ctx.block, ctx.kept, ctx.versions = block, kept, (block.w1_8.version, block.w2_8.version)
        return r

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dr):
        block, (y, z, n8, h8, stats, before, after) = ctx.block, ctx.kept
        x = ctx.saved_tensors[0]
        if (block.w1_8.version, block.w2_8.version) != ctx.versions:
            raise RuntimeError("the 8-bit weights have been set anew since the forward pass")
        n, width = x.shape
        hidden, dev, half = z.shape[1], x.device, torch.bfloat16
        dr = dr.contiguous()
        grads = {k: torch.empty_like(getattr(block, k)) for k in NAMES}
        # through the residual sum, the gate, the dropout and the norm after the block (the sum itself
        # passes dr on unchanged)
        dy = torch.empty_like(y)
        il.iris_block_norm_bwd(None, x, stats[1], after, dr=dr, y=y, dy=dy, dpost_w=grads["post_w"], dgate=grads["gate"])
        # the second product's bias: dy's column sums
        b2 = torch.empty(width, dtype=half, device=dev)
        il.iris_dropout(torch.empty_like(dy), dy, None, sums=b2)
        dy8, dy8_t, h8_t = il.iris_fp8_empty(n, width), il.iris_fp8_empty(width, n), il.iris_fp8_empty(hidden, n)
        il.iris_fp8_quantize(dy, dy8, dy8_t)
        il.iris_fp8_quantize(h8, None, h8_t)
        il.iris_fp8_mm(grads["w2"], dy8_t, h8_t)
        # back through the activation
        dz, b1 = torch.empty_like(z), torch.empty(hidden, dtype=half, device=dev)
        il.iris_fp8_mm_act_bwd(dz, dy8, block.w2_8.bwd, z, "gelu", dbias=b1)
        dz8, dz8_t, n8_t = il.iris_fp8_empty(n, hidden), il.iris_fp8_empty(hidden, n), il.iris_fp8_empty(width, n)
        il.iris_fp8_quantize(dz, dz8, dz8_t)
        il.iris_fp8_quantize(n8, None, n8_t)
        il.iris_fp8_mm(grads["w1"], dz8_t, n8_t)
        dn = torch.empty((n, width), dtype=half, device=dev)
        il.iris_fp8_mm(dn, dz8, block.w1_8.bwd)
        # the norm before the block; the stream's own gradient is added to it
        dx = torch.empty_like(x)
        il.iris_block_norm_bwd(dx, x, stats[0], before, dn=dn, dr=dr, dpre_w=grads["pre_w"])
        grads["b1"], grads["b2"] = b1.float(), b2.float()
        return (None, None, dx, *(grads[k] for k in NAMES))


class Block(torch.nn.Module):
    def __init__(self, width, hidden, p=0.1, alpha=1.0, device="cuda"):
        super().__init__()
        def param(t):
            return torch.nn.Parameter(t.to(device))
        self.w1, self.b1 = param(torch.randn(hidden, width) / width ** 0.5), param(0.1 * torch.randn(hidden))
        self.w2, self.b2 = param(torch.randn(width, hidden) / hidden ** 0.5), param(0.1 * torch.randn(width))
        self.pre_w, self.post_w, self.gate = param(torch.ones(width)), param(torch.ones(width)), param(torch.full((width,), 0.5))
        self.w1_8, self.w2_8 = Weight8(hidden, width), Weight8(width, hidden)
        self.p, self.alpha = p, alpha
        self.refresh()

    @torch.no_grad()
    def refresh(self):
        """After the weights have changed: their 8-bit copies."""
        self.w1_8.set(self.w1)
        self.w2_8.set(self.w2)

    def forward(self, x, dropout=None):
        """dropout: a il.Dropout of this step, or None (serving)."""
        if not torch.is_grad_enabled():
            return forward(self, x, dropout, False)[0]
        return BlockFunction.apply(self, dropout, x, *(getattr(self, k) for k in NAMES))


def train(tokens, width, hidden, steps, lr=0.02, seed=0):
    """Losses of `steps` gradient steps of two blocks towards two random ones."""
    torch.manual_seed(seed)
    blocks, goal = ([Block(width, hidden) for _ in range(2)] for _ in range(2))
    losses = []
    for step in range(steps):
        x = torch.randn(tokens, width, device="cuda")
        with torch.no_grad():
            target = goal[1](goal[0](x))
        for i, b in enumerate(blocks):
            # a mask of its own for every step and block
            x = b(x, il.Dropout(b.p, seed, offset=step * len(blocks) + i))
        loss = (x - target).square().mean()
        loss.backward()
        with torch.no_grad():
            for b in blocks:
                for w in b.parameters():
                    w -= lr * w.norm() / (w.grad.norm() + 1e-12) * w.grad
                    w.grad = None
                b.refresh()
        losses.append(loss.detach())
    return blocks, [float(v) for v in losses]


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--width", type=int, default=512)
    ap.add_argument("--hidden", type=int, default=1376)
    ap.add_argument("--steps", type=int, default=20)
    a = ap.parse_args()
    blocks, losses = train(a.tokens, a.width, a.hidden, a.steps)
    print("loss: " + " ".join(f"{v:.4f}" for v in losses))
    with torch.no_grad():
        x = torch.randn(1, a.width, device="cuda")
        for b in blocks:
            x = b(x)
    print(f"one token: output norm {float(x.norm()):.3f}")


if __name__ == "__main__":
    main()

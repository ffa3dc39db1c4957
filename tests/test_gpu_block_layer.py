"""The block operators together, as examples/fp8_block.py uses them: a residual block's
output and gradients against the same block in float64 on the CPU, the example, and a
captured step.

Tolerance, as for the 8-bit layer: an e4m3 rounding is 0.036 root-mean-square of a value,
a product of two rounded operands 0.051. What the block adds to the stream has passed
the roundings of n, W1, h and W2, two products' worth: sqrt(2) 0.051 = 0.072 (the norm
after it keeps relative errors; the norm before it and 16-bit roundings add under 0.003
each). The stream's part of r is exact. Gradients: dy comes from 32-bit dr by way of the
norm at a y that is off by 0.072; then up to three products with rounded operands
(dy W2; dz, W1; x8, dz_t) and h, z off by 0.051 again: at most seven such errors in
quadrature, 0.135. Compared in the 2-norm, with half as much again for what is not
uniform. The stream's gradient holds dr exactly beside the block's share.
"""
import importlib.util
import os
import sys

import pytest
import torch

import block_ref as bref
from gpu_util import note

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    spec = importlib.util.spec_from_file_location("fp8_block", os.path.join(ROOT, "examples", "fp8_block.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def rel(a, b):
    return float((a.double().cpu() - b).norm() / b.norm())


def norm64(v, w, eps=1e-6):
    return v * (v.square().mean(1, keepdim=True) + eps).rsqrt() * w


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,width,hidden,p", [(200, 256, 344, 0.2), (513, 384, 1376, 0.1), (33, 264, 200, 0.0), (1, 256, 344, 0.0)])
def test_block_and_gradients(tokens, width, hidden, p):
    ex = example()
    note(f"8-bit block {tokens} x {width} x {hidden}, p {p}")
    torch.manual_seed(tokens)
    block = ex.Block(width, hidden, p=p, alpha=0.7)
    with torch.no_grad():
        for k in ("pre_w", "post_w", "gate"):
            getattr(block, k).add_(0.2 * torch.randn(width, device="cuda"))
    x = torch.randn(tokens, width, device="cuda").requires_grad_()
    dr = torch.randn(tokens, width, device="cuda")
    drop = ex.il.Dropout(p, 77, 3) if p > 0 else None
    r = block(x, drop)
    r.backward(dr)
    xd = x.detach().double().cpu().requires_grad_()
    q = {k: getattr(block, k).detach().double().cpu().requires_grad_() for k in ex.NAMES}
    m = torch.from_numpy(bref.mask(tokens, width, p, 77, 3)) if p > 0 else 1.0
    z = norm64(xd, q["pre_w"]) @ q["w1"].t() + q["b1"]
    y = (z * torch.special.ndtr(z)) @ q["w2"].t() + q["b2"]
    rd = xd + 0.7 * q["gate"] * m * norm64(y, q["post_w"])
    rd.backward(dr.double().cpu())
    assert rel(r.detach() - x.detach(), (rd - xd).detach()) < 1.5 * 0.072
    assert rel(x.grad - dr, xd.grad - dr.double().cpu()) < 1.5 * 0.135
    for k in ex.NAMES:
        assert rel(getattr(block, k).grad, q[k].grad) < 1.5 * 0.135, k
    with torch.no_grad():
        serving = block(x, drop)
    assert torch.equal(serving, r), "what is kept for the backward pass changes nothing"


@pytest.mark.gpu
def test_example_runs_and_a_token_decodes():
    ex = example()
    note("8-bit block: training")
    blocks, losses = ex.train(128, 256, 344, 3)
    assert len(losses) == 3 and all(v == v for v in losses)
    with torch.no_grad():
        x = torch.randn(5, 256, device="cuda")
        many, one = blocks[0](x), blocks[0](x[3:4])
    assert torch.equal(many[3:4], one), "a row's result does not depend on the other rows"


@pytest.mark.gpu
def test_backward_refuses_weights_set_anew():
    ex = example()
    block = ex.Block(256, 344)
    x = torch.randn(20, 256, device="cuda").requires_grad_()
    r = block(x)
    block.refresh()
    with pytest.raises(RuntimeError, match="set anew"):
        r.backward(torch.ones_like(r))


@pytest.mark.gpu
def test_a_captured_decoding_step():
    """The serving path of two blocks in a graph, replayed with new tokens between eager work."""
    ex = example()
    torch.manual_seed(3)
    blocks = [ex.Block(512, 1376) for _ in range(2)]
    x = torch.randn(4, 512, device="cuda")

    def step():
        with torch.no_grad():
            return blocks[1](blocks[0](x))

    step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        out = step()
    for k in range(4):
        x.copy_(torch.randn(4, 512, device="cuda"))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, step()), k

"""examples/fp8_block.py between its passes: what its backward pass reads is either what
the forward pass read, or refused."""
import pytest
import torch

from gpu_util import note
from test_gpu_block_layer import example


def made(ex, p=0.3, counter=None):
    torch.manual_seed(5)
    block = ex.Block(256, 344, p=p)
    x = torch.randn(90, 256, device="cuda").requires_grad_()
    return block, x, ex.il.Dropout(p, 77, 3, counter), torch.randn(90, 256, device="cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["pre_w", "post_w", "gate", "x"])
def test_what_the_backward_pass_reads_may_not_change(name):
    ex = example()
    note(f"8-bit block: {name} changed between the passes")
    block, x, drop, dr = made(ex)
    r = block(x, drop)
    with torch.no_grad():
        (x if name == "x" else getattr(block, name)).mul_(2.0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        r.backward(dr)


@pytest.mark.gpu
@pytest.mark.parametrize("by", ["offset", "counter"])
def test_a_dropout_that_moves_on_keeps_the_earlier_masks(by):
    """Two forward passes with one handle that moves on between them, then their backward passes."""
    ex = example()
    note(f"8-bit block: two passes with one dropout, moved by its {by}")
    results = []
    for together in (False, True):
        counter = torch.zeros(1, dtype=torch.int64, device="cuda") if by == "counter" else None
        block, x, drop, dr = made(ex, counter=counter)
        outs = []
        for k in range(2):
            r = block(x, drop)
            if not together:
                r.backward(dr)
            outs.append(r)
            if by == "offset":
                drop.offset = drop.offset + 1
            else:
                counter.add_(1)
        if together:
            for r in outs:
                r.backward(dr)
        assert not torch.equal(outs[0], outs[1]), "a mask of its own for each pass"
        results.append([r.detach() for r in outs] + [x.grad] + [getattr(block, k).grad for k in ex.NAMES])
    assert all(torch.equal(a, b) for a, b in zip(*results))


@pytest.mark.gpu
def test_a_second_derivative_is_refused():
    """A loss with its gradient's norm in it: the gradient depends on x by way of dr and r, and has no derivative here."""
    ex = example()
    block, x, drop, dr = made(ex)
    loss = (block(x, drop) - dr).square().sum()
    (g,) = torch.autograd.grad(loss, x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (loss + g.square().sum()).backward()
    (g,) = torch.autograd.grad(block(x, drop), x, dr, create_graph=True)   # a given dr: nothing that a derivative could follow
    assert not g.requires_grad

"""The example's transformer block with its activations kept in 8 bits: its
gradients against the same block in binary64 and against those with the
activations as they are, and that its training steps run."""
import math

import pytest
import torch

from examples.block_step import Block, train
from tests.gpu_common import announce, device
from tests.test_gpu_block_example import cosine, reference

pytestmark = pytest.mark.gpu


def step(keep8, dev):
    m, width = 256, 512
    x = torch.randn((m, width), generator=torch.Generator().manual_seed(1)).bfloat16()
    at = torch.arange(m, device=dev)
    block = Block(width, 4, 2, 1024, 0.1, torch.where(at < 100, at, at - 100), (at >= 100).long(), seed=3, keep8=keep8)
    y, saved = block.forward(x.to(dev), 77)
    dy = torch.randn((m, width), generator=torch.Generator().manual_seed(2)).bfloat16()
    return block, x, y, dy, *block.backward(dy.to(dev), saved)


def test_block_gradients():
    """The forward pass does not read what is kept: the same bits. In 8 bits a
    value is off by at most 2^-4 of its size and 0.03 on average over its
    binade, a third of what E2M1 takes from the same operands, so the bounds of
    the block's test hold (0.78 counts 0.28 for each product; 0.28 and 0.03
    together are 0.282). Between the two ways the FP4 codes of the weights'
    gradients differ where a value was near a border between two codes: each
    side is within 0.28 sqrt(2) of the same product, 0.4 of its size at the
    worst for one product, a cosine of at least 1 / sqrt(1 + 0.4^2) = 0.92; the
    gradient of x passes the same FP4 products of the same gradients, and only
    SwiGLU's and the norms' factors differ, by up to 2^-4 each: three of them,
    0.19, a cosine of 0.98, on top of which stochastic rounding draws other
    codes (0.2 sqrt(2) for each of four products, 0.57: 0.86 in all)."""
    dev = device()
    announce("block gradients with activations in 8 bits")
    block, x, y, dy, dx, grad = step(True, dev)
    _, _, plain_y, _, plain_dx, plain = step(False, dev)
    assert torch.equal(y, plain_y)
    xr = x.double().requires_grad_()
    want, w = reference(block, xr, 77)
    want.backward(dy.double())
    assert cosine(dx, xr.grad) > 0.78 and cosine(dx, plain_dx) > 0.86
    for name, v in grad.items():
        assert cosine(v, w[name].grad) > 0.78, name
        assert cosine(v, plain[name]) > 0.86, name
        ratio = float(v.double().norm().cpu() / w[name].grad.norm())
        assert 0.6 < ratio < 1.6, (name, ratio)


def test_training_steps_run():
    dev = device()
    announce("example training steps with activations in 8 bits")
    args = dict(steps=3, tokens=256, width=512, hidden=1024, heads=4, kv_heads=2, device=dev, keep8=True)
    a, b = train(**args), train(**args)
    assert a == b and all(math.isfinite(v) for v in a)  # the same bits from the same seeds

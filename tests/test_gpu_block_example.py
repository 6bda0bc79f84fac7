"""The example's transformer block: its gradients against the same block in
binary64 with the same dropout masks, and its training steps."""
import math

import numpy as np
import pytest
import torch

from examples.block_step import Block, train
from tests import row_ref as R
from tests.gpu_common import B, announce, device

pytestmark = pytest.mark.gpu


def rms(x, g):
    return x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-5) * g


def reference(block, x, seed):
    """The block in binary64 on the CPU, from the bf16 weights it multiplies with."""
    w = {k: v.bfloat16().double().cpu().requires_grad_() for k, v in block.params.items()}
    m, width = x.shape
    n, d = block.heads + block.kv, block.dim
    t = rms(x, w["norm1"]) @ w["qkv"].T
    angle = block.positions.double().cpu()[:, None] * block.freq.double().cpu()
    c, s = angle.cos()[:, None], angle.sin()[:, None]
    h = t[:, :n * d].unflatten(1, (n, d))
    a, b = h[..., :d // 2], h[..., d // 2:]
    h = torch.cat([a * c - b * s, b * c + a * s], -1)
    q, k, v = h[:, :block.heads], h[:, block.heads:], t[:, n * d:].unflatten(1, (block.kv, d))
    rep = block.heads // block.kv
    k, v = k.repeat_interleave(rep, 1), v.repeat_interleave(rep, 1)
    at, seq = torch.arange(m), block.sequence.cpu()
    hidden = (at[None] > at[:, None]) | (seq[None] != seq[:, None])
    p = torch.softmax((torch.einsum("thd,shd->hts", q, k) / math.sqrt(d)).masked_fill(hidden, -math.inf), -1)
    o = torch.einsum("hts,shd->thd", p, v).flatten(1) @ w["o"].T

    def drop(z, stream):
        keep, scale = R.keep_mask(m, width, block.p, seed, stream)
        return z * torch.from_numpy(keep * np.float64(scale))

    h1 = x + drop(o, 0)
    f = block.hidden
    cc = (rms(h1, w["norm2"]) @ w["gate_up"].T).reshape(m, f // 32, 2, 32)
    g, u = cc[:, :, 0].reshape(m, f), cc[:, :, 1].reshape(m, f)
    return h1 + drop((torch.nn.functional.silu(g) * u) @ w["down"].T, 1), w


def cosine(a, b):
    a, b = a.detach().double().cpu().flatten(), b.detach().double().cpu().flatten()
    return float(a @ b / (a.norm() * b.norm()))


def test_block_gradients():
    """E2M1 with a scale per 32 is off by about 0.11 of a value's size, 0.16 to
    0.2 where it rounds stochastically; a product of two such operands by up
    to 0.28, and a gradient passes at most eight products in a row: 0.28
    sqrt(8) = 0.8 of its size at the worst, a cosine of at least
    1 / sqrt(1 + 0.8^2) = 0.78. A wrong sign, mask, order or factor anywhere
    gives far less on some parameter; the output, four products deep without
    stochastic rounding (0.16 sqrt(4) = 0.32) and mostly residual, 0.95."""
    dev = device()
    announce("block gradients")
    m, width = 256, 512
    x = torch.randn((m, width), generator=torch.Generator().manual_seed(1)).bfloat16()
    at = torch.arange(m, device=dev)
    block = Block(width, 4, 2, 1024, 0.1, torch.where(at < 100, at, at - 100), (at >= 100).long(), seed=3)
    y, saved = block.forward(x.to(dev), 77)
    dy = torch.randn((m, width), generator=torch.Generator().manual_seed(2)).bfloat16()
    dx, grad = block.backward(dy.to(dev), saved)
    xr = x.double().requires_grad_()
    want, w = reference(block, xr, 77)
    want.backward(dy.double())
    assert cosine(y, want) > 0.95
    assert cosine(dx, xr.grad) > 0.78
    for name, v in grad.items():
        assert v.shape == w[name].shape
        assert cosine(v, w[name].grad) > 0.78, name
        ratio = float(v.double().norm().cpu() / w[name].grad.norm())
        assert 0.6 < ratio < 1.6, (name, ratio)


def test_training_steps():
    dev = device()
    announce("example training steps")
    a = train(steps=6, tokens=256, width=512, hidden=1024, heads=4, kv_heads=2, device=dev)
    b = train(steps=6, tokens=256, width=512, hidden=1024, heads=4, kv_heads=2, device=dev)
    print(a)
    assert a == b  # the same bits from the same seeds
    assert all(math.isfinite(v) for v in a) and a[-1] < 0.98 * a[0]

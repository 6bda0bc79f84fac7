"""Row-wise operators at the edges of what they take: no rows, heads kept
apart from their tokens, outputs beside their inputs, launches wider than one
grid dimension, what overflows, and rows of NaN and Inf as an operand."""
import numpy as np
import pytest
import torch

from tests import row_ref as R
from tests.gpu_common import B, announce, device
from tests.test_gpu_row_ops import BF, F32, SEED, Padded, draw, same

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- no rows, no columns

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols", [(0, 64), (5, 0), (0, 0)])
def test_empty_matrices(rows, cols, dtype):
    """Every output that a call with rows gives comes out, empty."""
    dev = device()
    announce(f"empty matrices {rows}x{cols} {dtype}")
    e = torch.empty((rows, cols), dtype=dtype, device=dev)
    assert B.fp4_dropout(e, 0.5, seed=1, residual=e).shape == (rows, cols)
    for res, p in ((e, 0.0), (e, 0.1), (None, 0.1), (None, 0.0)):
        f = B.fp4_norm(e, residual=res, p=p, save=True)
        assert f.y.shape == (rows, cols) and f.mean.shape == f.rstd.shape == (rows,)
        assert (f.h is None) == (res is None and p == 0.0)
        h = e if f.h is None else f.h
        assert h.shape == (rows, cols) and h.dtype == dtype
        g = B.fp4_norm_grad(f.y, h, rstd=f.rstd, mean=f.mean, dres=res, p=p)
        assert g.dh.shape == (rows, cols) and g.dgamma.shape == g.dbeta.shape == (cols,)
        assert bool((g.dgamma == 0).all()) and bool((g.dbeta == 0).all())
        assert (g.dx is None) == (p == 0.0)
    if dtype == BF and rows == 0:
        for layout, k in ((B.LAYOUT_LINEAR, 64), (B.LAYOUT_TILED, 128)):
            z = torch.empty((0, k), dtype=BF, device=dev)
            f = B.fp4_norm(z, residual=z, mx=True, layout=layout)
            assert f.h.shape == (0, k) and (f.codes.shape, f.scales.shape) == B.mx_output_shapes(0, k, layout)
        dc, h = B.fp4_swiglu_grad_bf16(e, torch.empty((0, 2 * cols), dtype=BF, device=dev), want_h=True)
        assert dc.shape == (0, 2 * cols) and h.shape == (0, cols)
    freq = B.rotary_frequencies(16, device=dev)[0]
    for n, heads in ((0, 3), (4, 0)):
        x = torch.empty((n, heads, 32), dtype=dtype, device=dev)
        assert B.fp4_rotary(x, torch.zeros((n,), dtype=torch.int64, device=dev), freq).shape == (n, heads, 32)
    torch.cuda.synchronize()


# ---------------------------------------------------------------- heads of whole tokens

@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,heads,dim,rot", [(1, 3, 64, 64), (7, 1, 64, 32), (33, 5, 128, 128), (1030, 2, 100, 50), (9, 4, 48, 14)])
def test_rotary_of_heads_of_whole_tokens(n, heads, dim, rot, dtype, half):
    """[heads, tokens, dim] storage on either side and in place, at a pitch."""
    dev = device()
    announce(f"rotary of heads of whole tokens {dtype} {n}x{heads}x{dim} rot {rot} half {half}")
    style = B.ROTARY_HALF if half else B.ROTARY_INTERLEAVED
    x = draw((heads, n, dim), n + dim, dtype)
    pos = torch.randint(0, 1 << 18, (n,), generator=torch.Generator().manual_seed(n))
    freq, _ = B.rotary_frequencies(rot, 500000.0)
    args = dict(style=style, scale=1.25)
    want, e = R.rotary(x.transpose(0, 1).contiguous(), pos, freq, half, False, 1.25)
    px = Padded(heads, n * dim, dtype, dev, 24, 0, x.reshape(heads, -1))
    xv = px.view.unflatten(1, (n, dim)).transpose(0, 1)
    y = B.fp4_rotary(xv, pos.to(dev), freq.to(dev), **args)
    assert y.shape == (n, heads, dim) and y.is_contiguous()
    R.check(y, want, e, "y")
    py = Padded(heads, n * dim, dtype, dev, 5, 1)
    yv = py.view.unflatten(1, (n, dim)).transpose(0, 1)
    B.fp4_rotary(xv, pos.to(dev), freq.to(dev), y=yv, **args)
    same(yv, y, "into heads of whole tokens")
    assert py.untouched()
    B.fp4_rotary(xv, pos.to(dev), freq.to(dev), y=xv, **args)
    same(xv, y, "in place")
    assert px.untouched()

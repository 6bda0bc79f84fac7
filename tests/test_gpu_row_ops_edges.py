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


# ---------------------------------------------------------------- column blocks of one buffer

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols,gap", [(40, 64, 0), (37, 100, 3), (300, 1001, 0), (1100, 1032, 8), (20, 9000, 1)])
def test_outputs_in_other_columns_of_the_inputs_buffer(rows, cols, gap, dtype):
    dev = device()
    announce(f"column blocks of one buffer {rows}x{cols} gap {gap} {dtype}")
    n, step = 7, cols + gap
    buf = torch.full((rows, n * step), 777.0, dtype=dtype, device=dev)
    block = [buf[:, i * step:i * step + cols] for i in range(n)]
    ins = [draw((rows, cols), i, dtype).to(dev) for i in range(3)]
    g = (1 + draw((cols,), 4, F32, 0.2)).to(dev)

    def fill():
        buf.fill_(777.0)
        for b, v in zip(block, ins):
            b.copy_(v)

    def kept(written):
        m = torch.ones_like(buf, dtype=torch.bool)
        for i in (0, 1, 2, *written):
            m[:, i * step:i * step + cols] = False
        assert bool((buf[m] == 777.0).all())
        for b, v in zip(block, ins):
            same(b, v, "an input")

    want = B.fp4_dropout(ins[0], 0.1, seed=SEED, residual=ins[1])
    fill()
    B.fp4_dropout(block[0], 0.1, seed=SEED, residual=block[1], y=block[3])
    same(block[3], want, "dropout")
    kept((3,))
    want = B.fp4_norm(ins[0], g, residual=ins[1], p=0.1, seed=SEED, save=True)
    fill()
    B.fp4_norm(block[0], g, residual=block[1], p=0.1, seed=SEED, h=block[3], y=block[5])
    same(block[3], want.h, "h")
    same(block[5], want.y, "y")
    kept((3, 5))
    args = dict(mean=want.mean, rstd=want.rstd, p=0.1, seed=SEED)
    want = B.fp4_norm_grad(ins[0], ins[1], g, dres=ins[2], **args)
    fill()
    got = B.fp4_norm_grad(block[0], block[1], g, dres=block[2], dh=block[4], dx=block[6], **args)
    for a, b, what in zip(got, want, ("dh", "dx", "dgamma", "dbeta")):
        same(a, b, what)
    kept((4, 6))
    x = ins[0][:, :cols // 32 * 32].contiguous().unflatten(1, (-1, 32))
    freq, pos = B.rotary_frequencies(32, device=dev)[0], torch.arange(rows, device=dev)
    want = B.fp4_rotary(x, pos, freq)
    fill()
    v = [block[i][:, :cols // 32 * 32].unflatten(1, (-1, 32)) for i in (0, 3)]
    B.fp4_rotary(v[0], pos, freq, y=v[1])
    same(v[1], want, "rotary")
    kept((3,))


def test_swiglu_grad_in_other_columns_of_the_inputs_buffer():
    dev = device()
    announce("SwiGLU's gradient in column blocks of one buffer")
    for rows, f in ((33, 64), (300, 2048)):
        c, dh = draw((rows, 2 * f), 1, BF, 3.0).to(dev), draw((rows, f), 2, BF).to(dev)
        want = B.fp4_swiglu_grad_bf16(dh, c, want_h=True)
        buf = torch.full((rows, 7 * f), 777.0, dtype=BF, device=dev)
        vc, vd, vo, vh = buf[:, :2 * f], buf[:, 2 * f:3 * f], buf[:, 3 * f:5 * f], buf[:, 6 * f:]
        vc.copy_(c)
        vd.copy_(dh)
        B.fp4_swiglu_grad_bf16(vd, vc, dc=vo, h=vh)
        same(vo, want[0], "dc")
        same(vh, want[1], "h")
        same(vc, c, "c")
        same(vd, dh, "dh")
        assert bool((buf[:, 5 * f:6 * f] == 777.0).all())


# ---------------------------------------------------------------- errors

def test_out_of_memory_is_torchs_own_error():
    """The allocator refuses the output (its limit is lowered, the GPU has
    room): the caller gets torch's OutOfMemoryError, and goes on after it."""
    dev = device()
    announce("outputs that the allocator refuses")
    x = torch.zeros((4096, 8192), dtype=BF, device=dev)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    one, freq = torch.ones(4096, device=dev), B.rotary_frequencies(64, device=dev)[0]
    total = torch.cuda.get_device_properties(0).total_memory
    torch.cuda.set_per_process_memory_fraction((torch.cuda.memory_reserved() + (8 << 20)) / total)
    try:
        for call in (lambda: B.fp4_dropout(x, 0.1, seed=1), lambda: B.fp4_norm(x),
                     lambda: B.fp4_norm_grad(x, x, rstd=one, mean=one),
                     lambda: B.fp4_swiglu_grad_bf16(x[:, :4096], x),
                     lambda: B.fp4_rotary(x.view(4096, 128, 64), torch.zeros(4096, dtype=torch.int32, device=dev), freq),
                     lambda: B.fp4_dropout(x, 0.1, seed=1, stream=torch.cuda.Stream())):
            with pytest.raises(torch.OutOfMemoryError, match="allocate"):
                call()
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    assert torch.cuda.current_stream() == torch.cuda.default_stream()
    assert bool((B.fp4_dropout(x, 0.1, seed=1) == 0).all())


# ---------------------------------------------------------------- what overflows

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cols", [64, 1000, 4096, 6003])
def test_rows_whose_sums_overflow(cols, dtype):
    """As the header says: squares that sum to 2^128 give rstd 0 and y = beta,
    elements that do an infinite mean; other rows are left alone, and the
    gradient of such rows is 0 or NaN within them."""
    dev = device()
    announce(f"rows whose sums overflow, {cols} {dtype}")
    x = draw((5, cols), 1, dtype)
    x[1, cols // 2] = 1e30
    x[2] = 3e38
    x[3, 0], x[3, 1] = 1e19, -1e19  # squares 2e38: below 2^128
    b = draw((cols,), 2, dtype)
    for layer in (True, False):
        kind = B.NORM_LAYER if layer else B.NORM_RMS
        bd = b.to(dev)
        o = B.fp4_norm(x.to(dev), None, bd, kind=kind, save=True)
        assert o.rstd[1:3].tolist() == [0.0, 0.0]
        same(o.y[1], b, "y = beta")
        if layer:
            assert o.mean[2] == float("inf") and bool(torch.isnan(o.y[2]).all())
        else:
            same(o.y[2], b, "y = beta")
        y, _, rstd, ey, _, er = R.norm(x[[0, 3, 4]], None, b, layer, 1e-5)
        R.check(o.y[[0, 3, 4]], y, ey, "the other rows")
        R.check(o.rstd[[0, 3, 4]], rstd[:, 0], er[:, 0], "their rstd")
        dy = draw((5, cols), 3, dtype).to(dev)
        g = B.fp4_norm_grad(dy, x.to(dev), kind=kind, mean=o.mean, rstd=o.rstd, weights=False)
        alone = B.fp4_norm_grad(dy[[0, 3, 4]], x[[0, 3, 4]].to(dev), kind=kind, rstd=o.rstd[[0, 3, 4]],
                                mean=o.mean[[0, 3, 4]] if layer else None, weights=False)
        assert bool((g.dh[1] == 0).all())
        same(g.dh[[0, 3, 4]], alone.dh, "dh of the other rows")


def test_no_autograd():
    """An input may require grad; the outputs do not."""
    dev = device()
    announce("inputs that require grad")
    x = torch.randn((4, 64), device=dev).to(BF).requires_grad_()
    w = torch.ones(64, device=dev, requires_grad=True)
    for out in (B.fp4_dropout(x, 0.1, seed=1), B.fp4_norm(x, w).y,
                B.fp4_norm_grad(x, x, w, rstd=w[:4].detach(), mean=w[:4].detach()).dgamma,
                B.fp4_rotary(x[:, None], torch.arange(4, device=dev), w.detach()[:32])):
        assert not out.requires_grad and out.grad_fn is None

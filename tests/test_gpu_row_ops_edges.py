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


# ---------------------------------------------------------------- NaN and Inf in the fused operand

@pytest.mark.parametrize("cols,layout", [(64, 0), (96, 0), (512, 0), (8192, 0), (128, 1), (256, 1), (1024, 1), (4096, 1),
                                         (20480, 1)])
def test_operand_of_nan_and_inf_rows(cols, layout):
    """Byte for byte what the producer makes of y, NaN and Inf among it."""
    dev = device()
    announce(f"operand of NaN and Inf rows, {cols} layout {layout}")
    x = draw((37, cols), 1, BF)
    x[1, 3], x[2, cols - 1], x[3, 40], x[6, 5] = float("nan"), float("inf"), -float("inf"), 1e30
    x[4], x[5], x[7] = float("nan"), float("inf"), 3e38
    g = torch.ones(cols)
    g[7], g[9], g[33] = float("nan"), float("inf"), -float("inf")
    for kind in (B.NORM_LAYER, B.NORM_RMS):
        for w in (None, g.to(dev)):
            for res in (None, x.to(dev)):
                o = B.fp4_norm(x.to(dev), w, kind=kind, residual=res, mx=True, layout=layout)
                codes, scales = B.fp4_quantize_mx(o.y, layout=layout)
                assert torch.equal(o.codes, codes) and torch.equal(o.scales, scales)
                same(o.y, B.fp4_norm(x.to(dev), w, kind=kind, residual=res).y, "y")


# ---------------------------------------------------------------- in place at a pitch

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols,pad,lead", [(70, 100, 3, 1), (40, 1000, 24, 0), (33, 4096, 8, 0), (9, 5003, 5, 3),
                                                (700, 2056, 1, 1), (300, 9000, 3, 0), (20, 16392, 7, 1)])
def test_norm_and_gradient_in_place_at_a_pitch(rows, cols, pad, lead, dtype):
    """Results in the place of inputs whose rows lie apart; what lies between
    the rows is not touched."""
    dev = device()
    announce(f"norm and gradient in place {rows}x{cols} pad {pad} lead {lead} {dtype}")
    ins = [draw((rows, cols), i, dtype) for i in range(3)]
    g = (1 + draw((cols,), 4, F32, 0.2)).to(dev)

    def fresh():
        return [Padded(rows, cols, dtype, dev, pad, lead, v) for v in ins]

    d = [v.to(dev) for v in ins]
    want = B.fp4_dropout(d[0], 0.1, seed=SEED, residual=d[1])
    for i in (0, 1):
        t = fresh()
        B.fp4_dropout(t[0].view, 0.1, seed=SEED, residual=t[1].view, y=t[i].view)
        same(t[i].view, want, f"dropout in place {i}")
        assert all(v.untouched() for v in t)
    f = B.fp4_norm(d[0], g, residual=d[1], p=0.1, seed=SEED, save=True)
    for i, j in ((0, 1), (1, 0)):
        t = fresh()
        B.fp4_norm(t[0].view, g, residual=t[1].view, p=0.1, seed=SEED, h=t[i].view, y=t[j].view)
        same(t[i].view, f.h, f"h in place {i}")
        same(t[j].view, f.y, f"y in place {j}")
        assert all(v.untouched() for v in t)
    args = dict(mean=f.mean, rstd=f.rstd, p=0.1, seed=SEED)
    want = B.fp4_norm_grad(d[0], d[1], g, dres=d[2], **args)
    for weights in (True, False):
        for i, j in ((0, 1), (1, 2), (2, 0)):
            t = fresh()
            o = B.fp4_norm_grad(t[0].view, t[1].view, g, dres=t[2].view, dh=t[i].view, dx=t[j].view, weights=weights, **args)
            same(t[i].view, want.dh, f"dh in place {i}")
            same(t[j].view, want.dx, f"dx in place {j}")
            if weights:
                same(o.dgamma, want.dgamma, "dgamma")
                same(o.dbeta, want.dbeta, "dbeta")
            assert all(v.untouched() for v in t)


@pytest.mark.parametrize("M,F,pair,pad", [(33, 64, 32, 8), (70, 2048, 2048, 24), (300, 72, 8, 16), (9, 4104, 4104, 8)])
def test_swiglu_grad_in_place_at_a_pitch(M, F, pair, pad):
    dev = device()
    announce(f"SwiGLU's gradient in place {M}x{F} pair {pair} pad {pad}")
    c, dh = draw((M, 2 * F), 1, BF, 3.0), draw((M, F), 2, BF)
    want = B.fp4_swiglu_grad_bf16(dh.to(dev), c.to(dev), pair=pair, want_h=True)
    pc, pd = Padded(M, 2 * F, BF, dev, pad, 0, c), Padded(M, F, BF, dev, pad, 0, dh)
    B.fp4_swiglu_grad_bf16(pd.view, pc.view, pair=pair, dc=pc.view, h=pd.view)
    same(pc.view, want[0], "dc in place of c")
    same(pd.view, want[1], "h in place of dh")
    assert pc.untouched() and pd.untouched()


@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,heads,dim,rot,gap", [(33, 40, 128, 128, 1024), (7, 3, 80, 40, 8), (5, 2, 96, 36, 3),
                                                 (6, 5, 100, 50, 28), (1100, 3, 48, 48, 16), (9, 4, 24, 14, 1)])
def test_rotary_in_place_at_a_pitch(n, heads, dim, rot, gap, half, dtype):
    """As inside a fused QKV output: the elements from rot on, and what lies
    behind the heads, stay as they are."""
    dev = device()
    announce(f"rotary in place {dtype} {n}x{heads}x{dim} rot {rot} gap {gap} half {half}")
    x = draw((n, heads, dim), n + dim, dtype)
    pos = torch.randint(0, 1 << 18, (n,), generator=torch.Generator().manual_seed(n)).to(dev)
    args = dict(style=B.ROTARY_HALF if half else B.ROTARY_INTERLEAVED, scale=1.25)
    freq = B.rotary_frequencies(rot, 500000.0, device=dev)[0]
    want = B.fp4_rotary(x.to(dev), pos, freq, **args)
    p = Padded(n, heads * dim, dtype, dev, gap, 0, x.reshape(n, -1))
    v = p.view.unflatten(1, (heads, dim))
    assert not v.is_contiguous()
    B.fp4_rotary(v, pos, freq, y=v, **args)
    same(v, want, "in place")
    same(v[..., rot:], x[..., rot:], "elements from rot on")
    assert p.untouched()


# ---------------------------------------------------------------- far positions

@pytest.mark.parametrize("half", [True, False])
def test_rotary_positions_up_to_2_31(half):
    """Against sine and cosine of the angle's fraction of a turn, from integers:
    a frequency is f = m 2^-s exactly, and the position's product with it and
    the turns of 2 pi are taken at 200 bits. The kernel's own turns are off by
    2^-53 of themselves twice (the frequency over 2 pi, and its product with
    the position): at 2^31 positions and frequency 1, 2^31 / 2 pi 2^-52 turns,
    2^-21 radians."""
    from fractions import Fraction

    dev = device()
    announce(f"rotary at positions up to 2^31, half {half}")
    pos = [2 ** 29 - 3, 2 ** 30 + 1, 2 ** 31 - 1, -(2 ** 31), 2 ** 31 + 5]
    freq, _ = B.rotary_frequencies(64, 10000.0)
    # 2 pi to 200 bits, by Machin's formula
    one = 1 << 260

    def arctan_inverse(q):
        total, term, k = 0, one // q, 0
        while term:
            total += (-1) ** k * (term // (2 * k + 1))
            term //= q * q
            k += 1
        return total

    two_pi = Fraction(2 * 4 * (4 * arctan_inverse(5) - arctan_inverse(239)), one)
    angle = np.empty((len(pos), 32))
    for i, p in enumerate(pos):
        for j, f in enumerate(freq.double().tolist()):
            turns = Fraction(p) * Fraction(f) / two_pi
            angle[i, j] = float((turns - round(turns)) * two_pi)
    x = draw((len(pos), 2, 64), 1, F32)
    v = x.double().numpy()
    ia = np.arange(32) if half else 2 * np.arange(32)
    ib = ia + 32 if half else ia + 1
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    a, b = v[..., ia], v[..., ib]
    want, e = np.empty_like(v), np.empty_like(v)
    want[..., ia], want[..., ib] = a * c - b * s, b * c + a * s
    # row_ref.rotary's bound, and the turns
    e[..., ia] = e[..., ib] = (np.abs(a) + np.abs(b)) * (10 * R.U + 2.0 ** -20)
    style = B.ROTARY_HALF if half else B.ROTARY_INTERLEAVED
    R.check(B.fp4_rotary(x.to(dev), torch.tensor(pos, device=dev), freq.to(dev), style=style), want, e, "y")
    few = torch.tensor(pos[:4], dtype=torch.int32, device=dev)
    R.check(B.fp4_rotary(x[:4].to(dev), few, freq.to(dev), style=style), want[:4], e[:4], "y, 32-bit positions")


# ---------------------------------------------------------------- launches with a second grid dimension

def free_gib(dev):
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    return torch.cuda.mem_get_info(dev)[0] / 2 ** 30


def test_norm_past_2_20_workgroups():
    """2^24 + 77 rows of eight, sixteen to a workgroup, and 2^20 + 9 rows of a
    workgroup each: as the same rows in smaller calls, whose launches have one
    dimension."""
    dev = device()
    announce("norm past 2^20 workgroups")
    if free_gib(dev) < 24:
        pytest.skip("needs 24 GiB")
    for rows, cols in ((2 ** 24 + 77, 8), (2 ** 20 + 9, 1032)):
        g = torch.Generator(device=dev).manual_seed(1)
        x = torch.randn((rows, cols), generator=g, device=dev).to(BF)
        w = (1 + torch.randn((cols,), generator=g, device=dev) / 8).to(BF)
        whole = B.fp4_norm(x, w, save=True)
        grad = B.fp4_norm_grad(whole.y, x, w, mean=whole.mean, rstd=whole.rstd, weights=False).dh
        for lo in range(0, rows, rows // 5 + 1):
            part = slice(lo, min(rows, lo + rows // 5 + 1))
            o = B.fp4_norm(x[part], w, save=True)
            for a, b in ((whole.y[part], o.y), (whole.mean[part], o.mean), (whole.rstd[part], o.rstd)):
                assert torch.equal(a, b), (rows, cols, lo)
            d = B.fp4_norm_grad(o.y, x[part], w, mean=o.mean, rstd=o.rstd, weights=False).dh
            assert torch.equal(grad[part], d), (rows, cols, lo)


def test_norm_operand_past_2_20_workgroups():
    """The tiled operand, whose workgroups are permuted in runs of 256 rows."""
    dev = device()
    announce("norm's tiled operand past 2^20 workgroups")
    if free_gib(dev) < 24:
        pytest.skip("needs 24 GiB")
    rows, cols = 2 ** 20 + 300, 1152
    x = torch.randn((rows, cols), generator=torch.Generator(device=dev).manual_seed(2), device=dev).to(BF)
    o = B.fp4_norm(x, mx=True, layout=B.LAYOUT_TILED)
    codes, scales = B.fp4_quantize_mx(o.y, layout=B.LAYOUT_TILED)
    assert torch.equal(o.codes, codes) and torch.equal(o.scales, scales)


def test_rotary_past_2_20_workgroups():
    dev = device()
    announce("rotary past 2^20 workgroups")
    if free_gib(dev) < 24:
        pytest.skip("needs 24 GiB")
    n = 2 ** 27 + 1000  # one pair each, 128 to a workgroup
    x = torch.randn((n, 1, 2), generator=torch.Generator(device=dev).manual_seed(3), device=dev).to(BF)
    pos = torch.arange(n, dtype=torch.int32, device=dev)
    freq = torch.ones(1, device=dev)
    y = B.fp4_rotary(x, pos, freq)
    for lo in range(0, n, n // 5 + 1):
        part = slice(lo, min(n, lo + n // 5 + 1))
        assert torch.equal(y[part], B.fp4_rotary(x[part], pos[part], freq)), lo


def test_swiglu_grad_past_2_31_chunks():
    """2^28 + 40 rows of 64: rows at the start, around the second dimension's
    first and at the end, against calls on those rows alone. dc takes c's place
    (the rest of the memory holds whatever it holds)."""
    dev = device()
    announce("SwiGLU's gradient past 2^31 chunks")
    if free_gib(dev) < 160:
        pytest.skip("needs 160 GiB")
    rows, f = 2 ** 28 + 40, 64
    c = torch.empty((rows, 2 * f), dtype=BF, device=dev)
    dh = torch.empty((rows, f), dtype=BF, device=dev)
    for want_h in (False, True):
        want = []
        parts = [slice(0, 100), slice(2 ** 28 - 50, 2 ** 28 + 20), slice(rows - 10, rows)]
        for i, part in enumerate(parts):
            n = part.stop - part.start
            ci, di = draw((n, 2 * f), 2 * i, BF, 2.0).to(dev), draw((n, f), 2 * i + 1, BF).to(dev)
            c[part], dh[part] = ci, di
            want.append((ci, di))
        want = [B.fp4_swiglu_grad_bf16(di, ci, want_h=True) for ci, di in want]
        B.fp4_swiglu_grad_bf16(dh, c, dc=c, h=dh if want_h else None)
        for part, (dc, h) in zip(parts, want):
            assert torch.equal(c[part], dc)
            if want_h:
                assert torch.equal(dh[part], h)
    del c, dh
    torch.cuda.empty_cache()


# ---------------------------------------------------------------- sizes on either side of a rule

@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("n,heads,dim", [(8192, 2, 64), (4100, 3, 64), (2050, 2, 128), (20000, 1, 64), (1030, 6, 128), (5000, 4, 32)])
def test_rotary_few_heads(n, heads, dim, half):
    """Few heads, where a workgroup's tokens go by type and style: bf16 and
    binary32, against the binary64 form."""
    dev = device()
    announce(f"rotary of few heads {n}x{heads}x{dim} half {half}")
    pos = torch.randint(0, 1 << 18, (n,), generator=torch.Generator().manual_seed(n))
    freq, _ = B.rotary_frequencies(dim, 500000.0)
    for dtype in (BF, F32):
        x = draw((n, heads, dim), n + dim, dtype)
        want, e = R.rotary(x, pos, freq, half, False, 1.0)
        style = B.ROTARY_HALF if half else B.ROTARY_INTERLEAVED
        R.check(B.fp4_rotary(x.to(dev), pos.to(dev), freq.to(dev), style=style), want, e, "y")


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols", [(640, 8192), (641, 8192), (768, 7700), (769, 8192)])
def test_norm_grad_on_either_side_of_the_row_counts(rows, cols, dtype):
    """Weight sums beside the rows and in them, by type, in place too."""
    dev = device()
    announce(f"norm gradient {rows}x{cols} {dtype}")
    h, dy, dres = (draw((rows, cols), i, dtype, 2.0) for i in range(3))
    g = 1 + draw((cols,), 4, F32, 0.2)
    _, mean, rstd, _, _, _ = R.norm(h, g, None, True, 1e-5)
    mean, rstd = (torch.from_numpy(v[:, 0]).float() for v in (mean, rstd))
    dh, dg, db, edh, edg, edb = R.norm_grad(dy, h, g, mean, rstd, True, dres)
    args = dict(mean=mean.to(dev), rstd=rstd.to(dev))
    o = B.fp4_norm_grad(dy.to(dev), h.to(dev), g.to(dev), dres=dres.to(dev), **args)
    R.check(o.dh, dh, edh, "dh")
    R.check(o.dgamma, dg, edg, "dgamma")
    R.check(o.dbeta, db, edb, "dbeta")
    u = dy.to(dev)
    q = B.fp4_norm_grad(u, h.to(dev), g.to(dev), dres=dres.to(dev), dh=u, **args)
    for a, b in zip((u, q.dgamma, q.dbeta), (o.dh, o.dgamma, o.dbeta)):
        same(a, b, "in place")

"""The row-wise operators on the GPU (dropout, norm, its gradient, SwiGLU's
gradient, rotary positions) against their binary64 forms, within bounds that
row_ref.py derives; dropout and the fused MXFP4 operand bit for bit."""
import numpy as np
import pytest
import torch

from tests import row_ref as R
from tests.gpu_common import B, announce, device, synth

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
SEED = 0x5EEDCAFE12345


def draw(shape, seed, dtype, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


class Padded:
    """A matrix inside a wider poisoned buffer that starts `lead` elements in."""

    def __init__(self, rows, cols, dtype, dev, pad=0, lead=0, fill=None):
        self.buf = torch.full((lead + rows * (cols + pad) + 64,), 777.0, dtype=dtype, device=dev)
        self.view = torch.as_strided(self.buf, (rows, cols), (cols + pad, 1), lead)
        self.at = torch.as_strided(torch.arange(self.buf.numel(), device=dev), (rows, cols), (cols + pad, 1), lead)
        if fill is not None:
            self.view.copy_(fill)

    def untouched(self):
        m = torch.ones(self.buf.numel(), dtype=torch.bool, device=self.buf.device)
        m[self.at.reshape(-1)] = False
        return bool((self.buf[m] == 777.0).all())


def same(a, b, what):
    a, b = a.cpu(), b.cpu()
    w = torch.int16 if a.dtype == BF else torch.int32
    na, nb = torch.isnan(a), torch.isnan(b)
    assert torch.equal(na, nb), what
    assert torch.equal(a.contiguous().view(w)[~na], b.contiguous().view(w)[~nb]), what


SHAPES = [(1, 1), (3, 7), (2, 8), (5, 63), (33, 512), (17, 520), (9, 1000), (6, 1024), (5, 2048), (7, 2056), (4, 4096),
          (3, 5003), (2, 8192), (3, 8200), (2, 16384), (2, 16392), (2, 32768),
          (70, 100), (131, 128), (66, 136), (21, 200), (37, 256), (35, 257)]  # several rows to a wave, and not


# ---------------------------------------------------------------- dropout

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols,pad,lead", [(1, 1, 0, 0), (3, 5, 0, 0), (130, 8, 0, 0), (37, 1001, 0, 1),
                                                (64, 4096, 8, 0), (5, 2047, 3, 5)])
@pytest.mark.parametrize("p,res", [(0.0, True), (0.1, False), (0.5, True), (1.0, False)])
def test_dropout(dtype, rows, cols, pad, lead, p, res):
    dev = device()
    announce(f"dropout {dtype} {rows}x{cols} pad {pad} p {p} residual {res}")
    x, r = draw((rows, cols), 1, dtype), draw((rows, cols), 2, dtype) if res else None
    px = Padded(rows, cols, dtype, dev, pad, lead, x)
    pr = Padded(rows, cols, dtype, dev, pad + 1, lead, r) if res else None
    py = Padded(rows, cols, dtype, dev, pad, lead)
    B.fp4_dropout(px.view, p, seed=SEED, stream_id=3, residual=pr.view if res else None, y=py.view)
    same(py.view, R.dropout(x, r, p, SEED, 3), "y")
    assert py.untouched()


def test_dropout_rate_scale_and_streams():
    dev = device()
    announce("dropout's rate, unbiasedness, streams")
    n = 1 << 22
    x = torch.ones((n // 2048, 2048), device=dev)
    y = B.fp4_dropout(x, 0.3, seed=7)
    drop = round(0.3 * 65536)
    kept = float((y != 0).double().mean())
    q = 1 - drop / 65536
    assert abs(kept - q) < 5 * np.sqrt(q * (1 - q) / n)
    assert abs(float(y.double().mean()) - 1) < 5 * np.sqrt((1 - q) / q / n)
    other = B.fp4_dropout(x, 0.3, seed=7, stream_id=1)
    both = float(((y != 0) & (other != 0)).double().mean())
    assert abs(both - q * q) < 5 * np.sqrt(q * q / n)


def test_dropout_drops_nan_and_inf():
    dev = device()
    announce("dropout of NaN and Inf")
    x = torch.full((16, 64), float("nan"), dtype=BF)
    x[8:] = float("inf")
    y = B.fp4_dropout(x.to(dev), 0.5, seed=11)
    same(y, R.dropout(x, None, 0.5, 11), "y")
    assert bool((B.fp4_dropout(x.to(dev), 1.0, seed=11) == 0).all())


def test_dropout_in_place_and_its_gradient():
    dev = device()
    announce("dropout in place")
    x, r = draw((50, 333), 3, BF), draw((50, 333), 4, BF)
    want = B.fp4_dropout(x.to(dev), 0.25, seed=5, residual=r.to(dev))
    for which in (0, 1):
        t = [x.to(dev), r.to(dev)]
        B.fp4_dropout(t[0], 0.25, seed=5, residual=t[1], y=t[which])
        same(t[which], want, f"in place of argument {which}")
    # linear in x: the gradient is the same mask and scale
    dy = draw((50, 333), 5, F32)
    keep, scale = R.keep_mask(50, 333, 0.25, 5)
    same(B.fp4_dropout(dy.to(dev), 0.25, seed=5), torch.from_numpy(np.where(keep, dy.numpy() * scale, np.float32(0))), "dx")


def test_offsets_past_32_bits():
    dev = device()
    announce("row pitches whose offsets pass 2^32 elements")
    ld = 2 ** 31 - 5
    x, r = draw((4, 640), 6, BF), draw((4, 640), 7, BF)
    big = torch.empty((3 * ld + 640,), dtype=BF, device=dev)
    v = torch.as_strided(big, (4, 640), (ld, 1))
    v.copy_(x)
    want = R.dropout(x, r, 0.1, 9)
    same(B.fp4_dropout(v, 0.1, seed=9, residual=r.to(dev)), want, "dropout")
    o = B.fp4_norm(v, residual=r.to(dev), p=0.1, seed=9, kind=B.NORM_RMS, h=v)
    same(v, want, "norm's h, in place")
    y, _, _, ey, _, _ = R.norm(want, None, None, False, 1e-5)
    R.check(o.y, y, ey, "y")
    q = torch.as_strided(big, (4, 2, 64), (ld, 128, 1))
    q.copy_(draw((4, 2, 64), 8, BF))
    f, _ = B.rotary_frequencies(64)
    pos = torch.tensor([0, 5, 100000, 3])
    want, e = R.rotary(q.cpu(), pos, f, True, False, 1.0)
    R.check(B.fp4_rotary(q, pos.to(dev), f.to(dev)), want, e, "rotary")


# ---------------------------------------------------------------- norm

@pytest.mark.parametrize("layer", [True, False])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_norm(rows, cols, dtype, layer):
    dev = device()
    announce(f"norm {dtype} {rows}x{cols} layer {layer}")
    k = rows + cols
    for res, p, wt, pad, lead in [(False, 0.0, dtype, 0, 0), (True, 0.2, F32, 5, 1), (True, 0.0, BF, 8, 0),
                                  (False, 0.2, None, 0, 0)]:
        x, r = draw((rows, cols), k, dtype, 2.0), draw((rows, cols), k + 1, dtype) if res else None
        g = None if wt is None else 1 + draw((cols,), k + 2, F32, 0.2).to(wt)
        b = None if wt is None or not layer else draw((cols,), k + 3, wt, 0.3)
        px = Padded(rows, cols, dtype, dev, pad, lead, x)
        ph, py = Padded(rows, cols, dtype, dev, pad, lead), Padded(rows, cols, dtype, dev, pad, lead)
        o = B.fp4_norm(px.view, None if g is None else g.to(dev), None if b is None else b.to(dev),
                       kind=B.NORM_LAYER if layer else B.NORM_RMS, eps=1e-5, p=p, seed=SEED, stream_id=2, save=True,
                       residual=None if r is None else Padded(rows, cols, dtype, dev, pad + 3, lead, r).view,
                       h=ph.view, y=py.view)
        h = R.dropout(x, r, p, SEED, 2)
        same(ph.view, h, "h")
        y, mean, rstd, ey, em, er = R.norm(h, g, b, layer, 1e-5)
        R.check(o.y, y, ey, "y")
        R.check(o.rstd, rstd[:, 0], er[:, 0], "rstd")
        if layer:
            R.check(o.mean, mean[:, 0], em[:, 0], "mean")
        else:
            assert o.mean is None
        assert ph.untouched() and py.untouched()


@pytest.mark.parametrize("rows,cols,layout", [(1, 32, 0), (5, 96, 0), (45, 192, 0), (33, 4096, 0), (3, 1056, 0),
                                              (1, 128, 1), (70, 128, 1), (300, 256, 1), (33, 4096, 1),
                                              (31, 2176, 1), (64, 8320, 1), (2, 32768, 1), (40, 640, 1)])
@pytest.mark.parametrize("want_y", [True, False])
def test_norm_mx_operand(rows, cols, layout, want_y):
    dev = device()
    announce(f"norm with MXFP4 operand {rows}x{cols} layout {layout} y {want_y}")
    x = synth.activation(rows, cols, 77).to(dev)
    x[rows // 2] = 0  # a row of zero blocks
    g, b = (1 + draw((cols,), 1, F32, 0.2)).to(dev), draw((cols,), 2, F32, 0.1).to(dev)
    for kind, res in ((B.NORM_LAYER, True), (B.NORM_RMS, False)):
        cs, ss = B.mx_output_shapes(rows, cols, layout)
        codes, scales = (torch.full(s, 0xA5, dtype=torch.uint8, device=dev) for s in (cs, ss))
        args = dict(kind=kind, residual=x if res else None, p=0.1, seed=3)
        beta = b if kind == B.NORM_LAYER else None
        o = B.fp4_norm(x, g, beta, want_y=want_y, mx=True, layout=layout, codes=codes, scales=scales, **args)
        y = B.fp4_norm(x, g, beta, **args).y
        if want_y:
            same(o.y, y, "y")
        else:
            assert o.y is None
        wc, ws = B.fp4_quantize_mx(y, layout=layout)
        assert torch.equal(codes, wc) and torch.equal(scales, ws)


def test_norm_hard_rows():
    """A large mean, a constant row, zeros, one huge entry; a NaN or Inf row
    leaves the others alone."""
    dev = device()
    announce("norm's hard rows")
    for dtype in (BF, F32):
        for cols in (64, 1000, 4096):
            x = draw((7, cols), 5, dtype)
            x[0] += 4096.0
            x[1] = 3.0
            x[2] = 0.0
            x[3, cols // 2] = 1e30 if dtype == F32 else 1e15
            x[4, 0] = float("nan")
            x[5, cols - 1] = float("inf")
            for layer in (True, False):
                o = B.fp4_norm(x.to(dev), kind=B.NORM_LAYER if layer else B.NORM_RMS, save=True)
                keep = [0, 1, 2, 6] + ([3] if dtype == BF else [])
                y, _, rstd, ey, _, er = R.norm(x[keep], None, None, layer, 1e-5)
                R.check(o.y[keep], y, ey, f"y {dtype} {cols} {layer}")
                R.check(o.rstd[keep], rstd[:, 0], er[:, 0], "rstd")
                assert bool(torch.isnan(o.y[4]).all())
                assert bool(torch.isnan(o.y[5, -1]))


def test_norm_in_place():
    dev = device()
    announce("norm in place")
    for cols in (1000, 4096, 6003):
        x, r = draw((40, cols), 1, BF).to(dev), draw((40, cols), 2, BF).to(dev)
        g = draw((cols,), 3, BF).to(dev)
        want = B.fp4_norm(x, g, residual=r, p=0.1, seed=1, save=True)
        a, b = x.clone(), r.clone()
        got = B.fp4_norm(a, g, residual=b, p=0.1, seed=1, h=b, y=a)
        same(got.h, want.h, "h in place of residual")
        same(got.y, want.y, "y in place of x")


# ---------------------------------------------------------------- norm's gradient

GRAD_SHAPES = SHAPES + [(700, 129), (5000, 64), (40000, 16), (30000, 130), (1100, 1032), (600, 2100), (515, 9000), (660, 9000),
                        (641, 16392), (1030, 16392)]


@pytest.mark.parametrize("layer", [True, False])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols", GRAD_SHAPES)
def test_norm_grad(rows, cols, dtype, layer):
    dev = device()
    announce(f"norm gradient {dtype} {rows}x{cols} layer {layer}")
    k = 3 * rows + cols
    for res, p, wt, pad, lead in [(False, 0.0, dtype, 0, 0), (True, 0.2, F32, 5, 1), (True, 0.0, BF, 8, 0),
                                  (False, 0.2, None, 0, 0)]:
        h, dy = draw((rows, cols), k, dtype, 2.0), draw((rows, cols), k + 1, dtype)
        dres = draw((rows, cols), k + 2, dtype) if res else None
        g = None if wt is None else 1 + draw((cols,), k + 3, F32, 0.2).to(wt)
        _, mean, rstd, _, _, _ = R.norm(h, g, None, layer, 1e-5)
        mean, rstd = (torch.from_numpy(v[:, 0]).float() for v in (mean, rstd))
        pdh, pdx = Padded(rows, cols, dtype, dev, pad, lead), Padded(rows, cols, dtype, dev, pad + 1, lead)
        args = dict(kind=B.NORM_LAYER if layer else B.NORM_RMS, mean=mean.to(dev) if layer else None,
                    rstd=rstd.to(dev), p=p, seed=SEED, stream_id=4,
                    dres=None if dres is None else Padded(rows, cols, dtype, dev, pad + 3, lead, dres).view)
        pdy, phh = Padded(rows, cols, dtype, dev, pad, lead, dy), Padded(rows, cols, dtype, dev, pad + 2, lead, h)
        gd = None if g is None else g.to(dev)
        o = B.fp4_norm_grad(pdy.view, phh.view, gd, dh=pdh.view, dx=pdx.view if p > 0 else None, **args)
        dh, dg, db, edh, edg, edb = R.norm_grad(dy, h, g, mean, rstd, layer, dres)
        R.check(o.dh, dh, edh, "dh")
        R.check(o.dgamma, dg, edg, "dgamma")
        if layer:
            R.check(o.dbeta, db, edb, "dbeta")
        else:
            assert o.dbeta is None
        if p > 0:
            keep, scale = R.keep_mask(rows, cols, p, SEED, 4)
            f = keep * np.float64(scale)
            R.check(o.dx, dh * f, edh * f, "dx")
            assert pdx.untouched()
        assert pdh.untouched()
        again = B.fp4_norm_grad(pdy.view, phh.view, gd, **args)
        same(again.dgamma, o.dgamma, "the same bits again")
        if p == 0.0 and res:  # in place, and without the weights
            t = [pdy.view.clone(), phh.view.clone(), args["dres"].clone()]
            for i in range(3):
                u = [v.clone() for v in t]
                a = dict(args, dres=u[2])
                q = B.fp4_norm_grad(u[0], u[1], gd, weights=False, dh=u[i], **a)
                same(q.dh, o.dh, f"dh in place of argument {i}")
                assert q.dgamma is None and q.dbeta is None


@pytest.mark.parametrize("rows,cols", [(50, 5), (300, 1000), (700, 2048), (1500, 1032), (300, 9000), (260, 20000),
                                       (650, 9000), (650, 20000), (1030, 16392)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_norm_grad_in_place_with_weights(rows, cols, dtype):
    """dh or dx in the place of an input that the weight gradients are made
    from: every way of making them, small, in rows, and wide."""
    dev = device()
    announce(f"norm gradient in place with weights {rows}x{cols} {dtype}")
    t = [draw((rows, cols), i, dtype).to(dev) for i in range(3)]  # dy, h, dres
    g = (1 + draw((cols,), 4, F32, 0.2)).to(dev)
    f = B.fp4_norm(t[1], g, save=True)
    args = dict(mean=f.mean, rstd=f.rstd, p=0.1, seed=3)
    want = B.fp4_norm_grad(t[0], t[1], g, dres=t[2], **args)
    for i in range(3):
        for j in range(3):
            if i != j:
                u = [v.clone() for v in t]
                o = B.fp4_norm_grad(u[0], u[1], g, dres=u[2], dh=u[i], dx=u[j], **args)
                for a, b, what in zip(o, want, ("dh", "dx", "dgamma", "dbeta")):
                    same(a, b, f"{what}, dh in place {i}, dx in place {j}")


@pytest.mark.parametrize("rows,cols", [(650000, 5), (70001, 48), (3500, 1000), (1700, 2048), (1601, 2056), (400, 9000),
                                       (257, 14336), (170, 20000)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_norm_grad_without_weight_gradients(rows, cols, dtype):
    """Large calls without weight gradients: the rows' gradients are those of
    the call with them, bit for bit, in place too."""
    dev = device()
    announce(f"norm gradient without weight gradients {rows}x{cols} {dtype}")
    dy, h, dres = (draw((rows, cols), i, dtype).to(dev) for i in range(3))
    g = (1 + draw((cols,), 4, F32, 0.2)).to(dev)
    f = B.fp4_norm(h, g, save=True)
    for res, p in ((None, 0.0), (dres, 0.1)):
        args = dict(mean=f.mean, rstd=f.rstd, dres=res, p=p, seed=3)
        want = B.fp4_norm_grad(dy, h, g, **args)
        got = B.fp4_norm_grad(dy, h, g, weights=False, **args)
        assert got.dgamma is None and got.dbeta is None
        u = dy.clone()
        B.fp4_norm_grad(u, h, g, weights=False, dh=u, **args)
        same(got.dh, want.dh, "dh")
        same(u, want.dh, "dh in place")
        if p > 0:
            same(got.dx, want.dx, "dx")


def test_norm_grad_no_rows():
    dev = device()
    announce("norm gradient of no rows")
    e = torch.empty((0, 300), device=dev)
    z = torch.empty((0,), device=dev)
    o = B.fp4_norm_grad(e, e, rstd=z, mean=z, dgamma=torch.full((300,), 5.0, device=dev),
                        dbeta=torch.full((300,), 5.0, device=dev))
    assert bool((o.dgamma == 0).all()) and bool((o.dbeta == 0).all())


def test_norm_grad_nan_rows_and_columns():
    dev = device()
    announce("norm gradient with NaN")
    for rows, cols in ((40, 1024), (300, 2500)):
        h, dy = draw((rows, cols), 1, F32), draw((rows, cols), 2, F32)
        f = B.fp4_norm(h.to(dev), save=True)
        dy[3, 5] = float("nan")
        o = B.fp4_norm_grad(dy.to(dev), h.to(dev), mean=f.mean, rstd=f.rstd)
        bad = torch.isnan(o.dh).any(1).cpu()
        assert bad.tolist() == [i == 3 for i in range(rows)]
        assert torch.isnan(o.dgamma).nonzero().flatten().tolist() == [5]
        assert torch.isnan(o.dbeta).nonzero().flatten().tolist() == [5]


@pytest.mark.parametrize("layer", [True, False])
def test_norm_gradient_against_differences(layer):
    """d/dt of L(x + t v) = sum dy . y, by central differences of the kernel's
    own forward: L is off by at most sum |dy| ey (R.norm's bound) at each end,
    and the differences by t^2 / 6 of the third derivative, which for |v| <= 3
    and unit variance stays below 500 sum |dy| / cols per element of y."""
    dev = device()
    announce(f"norm gradient against differences, layer {layer}")
    rows, cols, t = 3, 257, 2.0 ** -8
    kind = B.NORM_LAYER if layer else B.NORM_RMS
    x, r, dy = draw((rows, cols), 1, F32), draw((rows, cols), 2, F32), draw((rows, cols), 3, F32)
    v = draw((rows, cols), 4, F32).clamp(-3, 3)
    g, b = 1 + draw((cols,), 5, F32, 0.2), draw((cols,), 6, F32)
    bd = b.to(dev) if layer else None

    def loss(x, r, g):
        o = B.fp4_norm(x.to(dev), g.to(dev), bd, kind=kind, residual=r.to(dev), p=0.25, seed=9)
        return float((o.y.double().cpu() * dy.double()).sum())

    f = B.fp4_norm(x.to(dev), g.to(dev), bd, kind=kind, residual=r.to(dev), p=0.25, seed=9, save=True)
    o = B.fp4_norm_grad(dy.to(dev), f.h, g.to(dev), kind=kind, mean=f.mean, rstd=f.rstd, p=0.25, seed=9)
    _, _, _, ey, _, _ = R.norm(f.h.cpu(), g, b if layer else None, layer, 1e-5)
    s = float(dy.abs().sum())
    noise = 2 * float((np.abs(dy.numpy()) * (ey + 4 * R.U)).sum()) / (2 * t)
    tol = noise + t * t / 6 * 500 * s / cols * 10 + 1e-5 * s
    for what, plus, minus, grad, along in [
            ("dx", (x + t * v, r, g), (x - t * v, r, g), o.dx, v), ("residual", (x, r + t * v, g), (x, r - t * v, g), o.dh, v),
            ("gamma", (x, r, g + t * v[0]), (x, r, g - t * v[0]), o.dgamma, v[0])]:
        num = (loss(*plus) - loss(*minus)) / (2 * t)
        ana = float((grad.double().cpu() * along.double()).sum())
        assert abs(num - ana) <= tol, (what, num, ana, tol)


# ---------------------------------------------------------------- SwiGLU's gradient

@pytest.mark.parametrize("M,F,pair,pad", [(1, 8, 8, 0), (5, 64, 32, 8), (3, 64, 64, 0), (17, 2080, 32, 16), (2, 14336, 32, 0),
                                          (9, 4104, 4104, 0), (70, 2048, 2048, 8), (300, 72, 8, 0)])
@pytest.mark.parametrize("want_h", [True, False])
def test_swiglu_grad(M, F, pair, pad, want_h):
    dev = device()
    announce(f"swiglu gradient {M}x{F} pair {pair} pad {pad}")
    c, dh = draw((M, 2 * F), 1, BF, 3.0), draw((M, F), 2, BF)
    pc, pd = Padded(M, 2 * F, BF, dev, pad, 0, c), Padded(M, F, BF, dev, pad, 0, dh)
    po, ph = Padded(M, 2 * F, BF, dev, pad, 0), Padded(M, F, BF, dev, pad, 0)
    B.fp4_swiglu_grad_bf16(pd.view, pc.view, pair=pair, dc=po.view, h=ph.view if want_h else None)
    dc, _, e = R.swiglu_grad(dh, c, pair)
    R.check(po.view, dc, e, "dc")
    assert po.untouched() and ph.untouched()
    if want_h:
        same(ph.view, B.fp4_swiglu_bf16(pc.view, F, pair=pair), "h as the forward writes it")
    u, w = pc.view.clone(), pd.view.clone()
    if pad == 0:
        q, k = B.fp4_swiglu_grad_bf16(w, u, pair=pair, dc=u, h=w)
        same(q, po.view, "dc in place of c")
        same(k, B.fp4_swiglu_bf16(pc.view, F, pair=pair), "h in place of dh")


def test_swiglu_grad_every_gate():
    dev = device()
    announce("swiglu gradient, every bf16 gate below 2^100")
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    g = bits.view(BF)
    g = g[torch.isfinite(g) & (g.float().abs() < 2.0 ** 100)]
    g = g[: g.numel() // 8 * 8]
    for uv, dv in ((1.0, 1.0), (-3.0, 0.0078125)):
        c = torch.cat([g, torch.full_like(g, uv)])[None]
        dh = torch.full((1, g.numel()), dv, dtype=BF)
        dc, _ = B.fp4_swiglu_grad_bf16(dh.to(dev), c.to(dev), pair=g.numel())
        want, _, e = R.swiglu_grad(dh, c, g.numel())
        R.check(dc, want, e, "dc")


def test_swiglu_gradient_against_differences():
    """Central differences of the binary64 definition: t^2 / 6 of the third
    derivative of SiLU (below 1) and the rounding of the difference."""
    dev = device()
    announce("swiglu gradient against differences")
    M, F, t = 4, 256, 2.0 ** -10
    c, dh = draw((M, 2 * F), 3, BF, 2.0), draw((M, F), 4, BF)
    dc, _ = B.fp4_swiglu_grad_bf16(dh.to(dev), c.to(dev), pair=F)
    g, u, d = c.double()[:, :F], c.double()[:, F:], dh.double()

    def h(g, u):
        return g / (1 + torch.exp(-g)) * u

    dg = d * (h(g + t, u) - h(g - t, u)) / (2 * t)
    du = d * (h(g, u + t) - h(g, u - t)) / (2 * t)
    want = torch.cat([dg, du], 1).numpy()
    err = np.abs(torch.cat([d * u, d], 1).numpy()) * (t * t / 6 + 1e-9) + R.swiglu_grad(dh, c, F)[2]
    R.check(dc, want, err, "dc")


# ---------------------------------------------------------------- rotary positions

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("n,heads,dim,rot,gap", [(1, 1, 2, 2, 0), (3, 5, 128, 128, 0), (33, 40, 128, 128, 1024), (7, 3, 80, 40, 8),
                                                 (5, 2, 96, 36, 3), (130, 1, 64, 64, 0), (9, 4, 256, 256, 0), (2, 3, 1024, 1024, 0),
                                                 (4, 2, 1000, 14, 5), (1100, 3, 48, 48, 0), (40000, 1, 64, 64, 0),
                                                 (6, 5, 100, 50, 0), (700, 3, 104, 100, 0), (6001, 3, 24, 24, 0)])
def test_rotary(n, heads, dim, rot, gap, half, dtype):
    dev = device()
    announce(f"rotary {dtype} {n}x{heads}x{dim} rot {rot} half {half}")
    style = B.ROTARY_HALF if half else B.ROTARY_INTERLEAVED
    x = draw((n, heads, dim), n + dim, dtype)
    px = Padded(n, heads * dim, dtype, dev, gap, 0, x.reshape(n, -1))
    py = Padded(n, heads * dim, dtype, dev, gap + 1, 1)
    xv, yv = (p.view.unflatten(1, (heads, dim)) for p in (px, py))
    pos = torch.randint(0, 1 << 20, (n,), generator=torch.Generator().manual_seed(n))
    pos[0] = 0
    pos[-1] = -17
    freq, _ = B.rotary_frequencies(rot, 500000.0)
    for inverse, scale, pt in ((False, 1.0, torch.int64), (True, 1.25, torch.int32)):
        B.fp4_rotary(xv, pos.to(pt).to(dev), freq.to(dev), style=style, inverse=inverse, scale=scale, y=yv)
        want, e = R.rotary(x, pos, freq, half, inverse, scale)
        R.check(yv, want, e, "y")
        assert py.untouched()
        z = xv.clone()
        B.fp4_rotary(z, pos.to(dev), freq.to(dev), style=style, inverse=inverse, scale=scale, y=z)
        same(z, yv, "in place")


def test_rotary_far_positions():
    dev = device()
    announce("rotary at positions up to 2^31")
    pos = torch.tensor([2 ** 20, 2 ** 24 + 1, 2 ** 29 - 3])
    freq, _ = B.rotary_frequencies(128)
    x = draw((3, 2, 128), 1, F32)
    want, e = R.rotary(x, pos, freq, True, False, 1.0)
    # binary64's 53 bits at 2^29 positions: 2^-53 2^29 radians and the same from 1 / 2 pi
    e = e + (np.abs(x.numpy()).max() * 2) * 2.0 ** -22
    R.check(B.fp4_rotary(x.to(dev), pos.to(dev), freq.to(dev)), want, e, "y")


def test_rotary_scores_depend_on_distance_only():
    dev = device()
    announce("rotary's defining property")
    q, k = draw((1, 1, 64), 1, F32), draw((1, 1, 64), 2, F32)
    f = B.rotary_frequencies(64)[0].to(dev)
    s = []
    for base in (0, 1000, 123456):
        a = B.fp4_rotary(q.to(dev), torch.tensor([base + 7], device=dev), f)
        b = B.fp4_rotary(k.to(dev), torch.tensor([base], device=dev), f)
        s.append(float((a.double() * b.double()).sum()))
    bound = 2 * 64 * 4 * 16 * R.U * float(q.abs().max() * k.abs().max())
    assert abs(s[0] - s[1]) < bound and abs(s[0] - s[2]) < bound


# ---------------------------------------------------------------- streams and graphs

def test_side_stream_and_graph():
    dev = device()
    announce("row operators on a side stream and in a graph")
    rows, cols = 512, 2048
    x, r = draw((rows, cols), 1, BF).to(dev), draw((rows, cols), 2, BF).to(dev)
    g = draw((cols,), 3, F32).to(dev)
    f = B.rotary_frequencies(128)[0].to(dev)
    pos = torch.arange(rows, device=dev)
    ws = torch.empty((B.lib().fp4q_norm_grad_workspace_bytes(rows, cols),), dtype=torch.uint8, device=dev)

    def step():
        o = B.fp4_norm(x, g, residual=r, p=0.1, seed=1, save=True, mx=True)
        d = B.fp4_norm_grad(o.y, o.h, g, mean=o.mean, rstd=o.rstd, p=0.1, seed=1, workspace=ws)
        q = B.fp4_rotary(d.dx.unflatten(1, (16, 128)), pos, f)
        s, h = B.fp4_swiglu_grad_bf16(B.fp4_dropout(r, 0.2, seed=2)[:, :1024].contiguous(), d.dh, want_h=True)
        return [o.y, o.codes, o.scales, d.dh, d.dx, d.dgamma, d.dbeta, q, s, h]

    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(3):
        x.copy_(draw((rows, cols), 10 + k, BF).to(dev))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        assert all(torch.equal(a, b) for a, b in zip(got, step())), k
        torch.cuda.synchronize()


@pytest.mark.parametrize("rows", [100, 1200])
def test_named_stream(rows):
    """`stream`: every operator on it, its outputs, workspace (the larger size
    needs one) and results as on the current one."""
    dev = device()
    announce(f"row operators on a stream of their own, {rows} rows")
    side, cols = torch.cuda.Stream(), 1024
    x, r, dy = (draw((rows, cols), i, BF).to(dev) for i in range(3))
    c = draw((rows, 2 * cols), 3, BF).to(dev)
    gamma = (1 + draw((cols,), 4, F32, 0.2)).to(dev)
    pos = torch.arange(rows, device=dev)
    freq = B.rotary_frequencies(64, device=dev)[0]

    def step(**s):
        d = B.fp4_dropout(x, 0.2, seed=3, residual=r, **s)
        f = B.fp4_norm(x, gamma, residual=r, p=0.2, seed=4, save=True, mx=True, **s)
        g = B.fp4_norm_grad(dy, f.h, gamma, mean=f.mean, rstd=f.rstd, p=0.2, seed=4, **s)
        return [d, *f, *g, *B.fp4_swiglu_grad_bf16(dy, c, want_h=True, **s),
                B.fp4_rotary(x.view(rows, 8, 128), pos, freq, **s)]

    want = step()
    torch.cuda.synchronize()
    got = step(stream=side)
    side.synchronize()
    for i, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(a, b), f"output {i}"
    with pytest.raises(ValueError, match="2-D"):
        B.fp4_norm_grad(dy[0], x[0], rstd=gamma, stream=side)


def test_refusals_reach_the_caller():
    dev = device()
    announce("row operators' refusals through the binding (nothing is launched)")
    x = torch.zeros((4, 64), dtype=BF, device=dev)
    v = torch.zeros((4,), device=dev)
    for call, status in ((lambda: B.fp4_dropout(x, 1.5, seed=1), B.EINVAL), (lambda: B.fp4_norm(x, kind=7), B.EINVAL),
                         (lambda: B.fp4_norm(x, kind=B.NORM_RMS, mean=v), B.EINVAL),
                         (lambda: B.fp4_norm_grad(x, x, rstd=v), B.EINVAL),  # a layer norm without its means
                         (lambda: B.fp4_swiglu_grad_bf16(x, torch.zeros((4, 128), dtype=BF, device=dev), pair=12), B.ESHAPE),
                         (lambda: B.fp4_rotary(x[:, None], torch.zeros((4,), dtype=torch.int32, device=dev),
                                               torch.zeros((40,), device=dev)), B.ESHAPE)):
        with pytest.raises(B.Fp4qError) as e:
            call()
        assert e.value.status == status
    for call in (lambda: B.fp4_dropout(x, 0.1, seed=1, y=x.cpu()), lambda: B.fp4_dropout(x, 0.1, seed=1, residual=x[:3]),
                 lambda: B.fp4_norm(x, v), lambda: B.fp4_norm_grad(x, x, rstd=v.double()),
                 lambda: B.fp4_rotary(x[:, None], v, v)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        B.fp4_dropout(x, "half", seed=1)
    torch.cuda.synchronize()

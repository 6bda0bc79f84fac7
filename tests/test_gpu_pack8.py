"""8-bit block-scaled rows on the GPU: packing and unpacking bit for bit as the
plain form, the packing norm as norm and packing, the gradients as those of the
unpacked rows and against binary64 within bounds that row_ref.py derives."""
import math

import numpy as np
import pytest
import torch

from tests import pack8_ref as P
from tests import row_ref as R
from tests.gpu_common import B, announce, device
from tests.test_gpu_row_ops import Padded, draw, same

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def bytes_equal(got, want, what):
    got, want = [np.asarray(t.cpu() if isinstance(t, torch.Tensor) else t) for t in (got, want)]
    assert got.shape == want.shape, what
    bad = np.argwhere(got != want)
    assert not len(bad), f"{what}: {len(bad)} of {got.size} differ, first at {bad[0]}: {got[tuple(bad[0])]} for {want[tuple(bad[0])]}"


class Bytes:
    """8-bit rows inside poisoned buffers, the scales at an odd address."""

    def __init__(self, rows, cols, dev):
        self.bufs = [torch.full((32 + n + 64,), 0xA5, dtype=torch.uint8, device=dev) for n in (rows * cols, rows * cols // 32)]
        self.codes = self.bufs[0][16:16 + rows * cols].view(rows, cols)
        self.scales = self.bufs[1][17:17 + rows * cols // 32].view(rows, cols // 32)

    def untouched(self):
        return all(bool((b[:lead] == 0xA5).all()) and bool((b[lead + t.numel():] == 0xA5).all())
                   for b, t, lead in zip(self.bufs, (self.codes, self.scales), (16, 17)))


def wide_range(rows, cols, seed, dtype):
    """Values over many binades, a few zeros among them."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((rows, cols), generator=g)
    x = x * torch.exp2(torch.randint(-20, 21, (rows, cols), generator=g).float())
    x[torch.rand((rows, cols), generator=g) < 0.02] = 0
    return x.to(dtype)


# ---------------------------------------------------------------- packing

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols,pad,lead", [(1, 32, 0, 0), (3, 32, 1, 1), (1, 4096, 0, 0), (37, 96, 0, 0),
                                                (65, 1056, 8, 8), (130, 2048, 3, 5), (129, 8224, 0, 1)])
def test_pack_and_unpack(dtype, rows, cols, pad, lead):
    dev = device()
    announce(f"pack8 {dtype} {rows}x{cols} pad {pad}")
    x = wide_range(rows, cols, rows + cols, dtype)
    px, out = Padded(rows, cols, dtype, dev, pad, lead, x), Bytes(rows, cols, dev)
    B.fp4_pack8(px.view, codes=out.codes, scales=out.scales)
    codes, scales = P.pack8(x)
    bytes_equal(out.scales, scales, "scales")
    bytes_equal(out.codes, codes, "codes")
    assert out.untouched()
    made = B.fp4_pack8(px.view)
    assert torch.equal(made[0], out.codes) and torch.equal(made[1], out.scales)
    py = Padded(rows, cols, dtype, dev, pad, lead)
    B.fp4_unpack8(out.codes, out.scales, y=py.view)
    same(py.view, torch.from_numpy(P.values(codes, scales)).to(dtype), "values")
    assert py.untouched()
    same(B.fp4_unpack8(out.codes, out.scales, out_dtype=dtype), py.view, "values made")


def test_every_bf16_value():
    """Each bf16 pattern alone in its block, and beside a one: NaN, infinities, subnormals, the largest."""
    dev = device()
    announce("pack8 of every bf16 value")
    every = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(BF)
    x = torch.zeros((65536, 64), dtype=BF)
    x[:, 7] = every
    x[:, 32 + 31] = every
    x[:, 32] = 1.0
    codes, scales = P.pack8(x)
    got = B.fp4_pack8(x.to(dev))
    bytes_equal(got[1], scales, "scales")
    bytes_equal(got[0], codes, "codes")
    wide = B.fp4_pack8(x.float().to(dev))
    assert torch.equal(wide[0], got[0]) and torch.equal(wide[1], got[1])
    same(B.fp4_unpack8(*got, out_dtype=F32), torch.from_numpy(P.values(codes, scales)).float(), "values")
    # (values in binary32 are exact; bf16 rounds below 2^-120 only)
    same(B.fp4_unpack8(*got), torch.from_numpy(P.values(codes, scales)).float().to(BF), "bf16 values")
    back = B.fp4_unpack8(*got).float().cpu()
    finite = x.isfinite()
    assert bool(back[finite].isfinite().all()) and bool(back[~finite].isnan().all())


def test_binary32_rounding():
    """Binary32 on and beside E4M3's midpoints, the largest magnitudes, and subnormal blocks."""
    dev = device()
    announce("pack8 of binary32 edges")
    mid = torch.from_numpy(P.MIDDLE).float()
    v = torch.cat([mid, torch.nextafter(mid, torch.tensor(math.inf)), torch.nextafter(mid, torch.tensor(0.0))])
    v = torch.cat([v, -v])[:704]
    x = torch.zeros((len(v) // 22 + 1, 32))
    x[:, 31] = 448
    x[:len(v) // 22, :22] = v[:len(v) // 22 * 22].view(-1, 22)
    for scale in (1.0, 2.0 ** -40, 2.0 ** 118):
        y = x * scale
        codes, scales = P.pack8(y)
        got = B.fp4_pack8(y.to(dev))
        bytes_equal(got[1], scales, "scales")
        bytes_equal(got[0], codes, "codes")
    top = torch.finfo(F32).max
    rows = [[top, -top, top / 2], [2.0 ** -149, 0.0, -(2.0 ** -149)], [2.0 ** -126, 2.0 ** -130, 0.0],
            [448.0, 464.0, 447.9], [448.00003, -448.00003, 1.0], [math.inf, -math.inf, top], [math.nan, 448.0, -3.0],
            [1.75 * 2.0 ** 127, 1.9375 * 2.0 ** 127, -1.0], [-0.0, 0.0, -0.0], [math.nan, math.inf, -math.inf]]
    x = torch.zeros((len(rows), 32))
    x[:, 5:8] = torch.tensor(rows)
    codes, scales = P.pack8(x)
    got = B.fp4_pack8(x.to(dev))
    bytes_equal(got[1], scales, "scales")
    bytes_equal(got[0], codes, "codes")


@pytest.mark.parametrize("rows,cols", [(0, 64), (3, 0), (0, 0)])
def test_empty(rows, cols):
    dev = device()
    announce(f"pack8 of {rows}x{cols}")
    x = torch.zeros((rows, cols), dtype=BF, device=dev)
    codes, scales = B.fp4_pack8(x)
    assert codes.shape == (rows, cols) and scales.shape == (rows, cols // 32)
    assert B.fp4_unpack8(codes, scales).shape == (rows, cols)
    o = B.fp4_norm_pack8(x, want_y=True)
    assert o.codes8.shape == (rows, cols) and o.y.shape == (rows, cols)
    g = B.fp4_norm_grad_pack8(x, codes, scales, rstd=torch.ones(rows, device=dev), mean=torch.ones(rows, device=dev))
    assert g.dh.shape == (rows, cols) and bool((g.dgamma == 0).all())


def test_offsets_past_32_bits():
    dev = device()
    announce("pack8 past 2^32 bytes of codes")
    rows, cols = (1 << 17) + 3, 1 << 15
    x = torch.zeros((rows, cols), dtype=BF, device=dev)
    x[0], x[-1] = wide_range(1, cols, 1, BF)[0].to(dev), wide_range(1, cols, 2, BF)[0].to(dev)
    codes, scales = B.fp4_pack8(x)
    for i in (0, -1):
        want = P.pack8(x[i:i + 1 or None].cpu())
        bytes_equal(codes[i:i + 1 or None], want[0], "codes")
        bytes_equal(scales[i:i + 1 or None], want[1], "scales")
    assert int(codes[1:-1].max()) == 0
    del x
    y = B.fp4_unpack8(codes, scales)
    for i in (0, -1):
        same(y[i], B.fp4_unpack8(codes[i:i + 1 or None].contiguous(), scales[i:i + 1 or None].contiguous())[0], "values")


# ---------------------------------------------------------------- the packing norm

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows,cols", [(1, 32), (5, 32), (70, 96), (131, 128), (37, 256), (33, 512), (17, 544), (6, 1024),
                                       (5, 2048), (1, 4096), (7, 4096), (3, 5024), (3, 8224), (2, 16384), (2, 16416),
                                       (2, 32768)])
def test_norm_pack8(rows, cols, dtype):
    dev = device()
    k = rows + cols
    announce(f"packing norm {dtype} {rows}x{cols}")
    for layer, res, p, gamma in ((True, True, 0.1, True), (False, True, 0.0, True), (False, False, 0.0, False)):
        x, r = draw((rows, cols), k, dtype, 3.0).to(dev), draw((rows, cols), k + 1, dtype).to(dev)
        w = (1 + draw((cols,), k + 2, F32, 0.2)).to(dev) if gamma else None
        b = draw((cols,), k + 3, F32).to(dev) if layer else None
        args = dict(kind=B.NORM_LAYER if layer else B.NORM_RMS, residual=r if res else None, p=p, seed=9, save=True)
        want = B.fp4_norm(x, w, b, **args)
        c8, s8 = B.fp4_pack8(want.y)
        out = Bytes(rows, cols, dev)
        got = B.fp4_norm_pack8(x, w, b, codes8=out.codes, scales8=out.scales, want_y=True, **args)
        bytes_equal(got.scales8, s8, "scales8")
        bytes_equal(got.codes8, c8, "codes8")
        assert out.untouched()
        for name in ("y", "h", "mean", "rstd"):
            a, c = getattr(got, name), getattr(want, name)
            assert (a is None) == (c is None), name
            if a is not None:
                same(a, c, name)
        lone = B.fp4_norm_pack8(x, w, b, **args)
        assert lone.y is None and torch.equal(lone.codes8, c8) and torch.equal(lone.scales8, s8)


@pytest.mark.parametrize("rows,cols,layout", [(1, 128, B.LAYOUT_TILED), (33, 4096, B.LAYOUT_TILED), (40, 96, B.LAYOUT_LINEAR),
                                              (300, 256, B.LAYOUT_TILED), (5, 8192, B.LAYOUT_LINEAR)])
def test_norm_pack8_beside_the_operand(rows, cols, layout):
    dev = device()
    announce(f"packing norm beside the MXFP4 operand {rows}x{cols} layout {layout}")
    x, r = draw((rows, cols), 5, BF).to(dev), draw((rows, cols), 6, BF).to(dev)
    want = B.fp4_norm(x, residual=r, mx=True, layout=layout)
    c8, s8 = B.fp4_pack8(want.y)
    got = B.fp4_norm_pack8(x, residual=r, mx=True, layout=layout)
    assert got.y is None
    for a, b in ((got.codes, want.codes), (got.scales, want.scales), (got.h, want.h), (got.codes8, c8), (got.scales8, s8)):
        assert torch.equal(a, b)


def test_norm_pack8_of_nan_and_inf_rows():
    dev = device()
    announce("packing norm of NaN and Inf rows")
    x = draw((6, 256), 1, BF)
    x[1, 3], x[2, 5], x[3, 7], x[4] = math.nan, math.inf, -math.inf, 0
    o = B.fp4_norm_pack8(x.to(dev), kind=B.NORM_RMS, want_y=True)
    want = B.fp4_pack8(o.y)
    assert torch.equal(o.codes8, want[0]) and torch.equal(o.scales8, want[1])
    v = B.fp4_unpack8(o.codes8, o.scales8)
    assert bool(v[1].isnan().all()) and bool(v[[0, 4, 5]].isfinite().all())


def test_norm_pack8_in_place():
    dev = device()
    announce("packing norm in place")
    x, r = draw((50, 320), 3, BF), draw((50, 320), 4, BF)
    want = B.fp4_norm_pack8(x.to(dev), residual=r.to(dev), p=0.2, seed=1, want_y=True)
    tx, tr = x.to(dev), r.to(dev)
    got = B.fp4_norm_pack8(tx, residual=tr, p=0.2, seed=1, h=tr, y=tx)
    assert torch.equal(tx, want.y) and torch.equal(tr, want.h)
    assert torch.equal(got.codes8, want.codes8) and torch.equal(got.scales8, want.scales8)


# ---------------------------------------------------------------- the gradients

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layer", [True, False])
@pytest.mark.parametrize("rows,cols", [(1, 32), (70, 96), (131, 128), (37, 256), (9, 512), (1000, 1024), (5, 2048), (4, 4096),
                                       (900, 4096), (3, 5024), (700, 8192), (2, 16384), (700, 12000), (2, 16416),
                                       (1100, 16416), (2, 32768)])
def test_norm_grad_pack8(rows, cols, dtype, layer):
    """Every bit as the gradient of the rows unpacked; and within the bounds of the formula in binary64."""
    dev = device()
    k = 3 * rows + cols
    announce(f"norm gradient of 8-bit rows {dtype} {rows}x{cols} layer {layer}")
    h, dy = draw((rows, cols), k, dtype, 2.0).to(dev), draw((rows, cols), k + 1, dtype).to(dev)
    dres = draw((rows, cols), k + 2, dtype).to(dev)
    gamma = (1 + draw((cols,), k + 3, F32, 0.2)).to(dev)
    kind = B.NORM_LAYER if layer else B.NORM_RMS
    f = B.fp4_norm(h, gamma, kind=kind, save=True)
    codes, scales = B.fp4_pack8(h)
    values = B.fp4_unpack8(codes, scales, out_dtype=dtype)
    same(values.double().cpu().to(dtype), torch.from_numpy(P.values(codes.cpu(), scales.cpu())).to(dtype), "values")
    for res, p, w, sums in ((True, 0.1, gamma, True), (False, 0.0, gamma, True), (True, 0.0, None, False)):
        args = dict(kind=kind, mean=f.mean, rstd=f.rstd, dres=dres if res else None, p=p, seed=5, weights=sums)
        want = B.fp4_norm_grad(dy, values, w, **args)
        got = B.fp4_norm_grad_pack8(dy, codes, scales, w, **args)
        for name in ("dh", "dx", "dgamma", "dbeta"):
            a, b = getattr(got, name), getattr(want, name)
            assert (a is None) == (b is None), name
            if a is not None:
                same(a, b, f"{name}, p {p}")
    if rows * cols <= 1 << 20:
        dh, dg, db, eh, eg, eb = R.norm_grad(dy.cpu(), values.cpu(), gamma.cpu(), f.mean.cpu() if layer else None,
                                             f.rstd.cpu(), layer, dres.cpu())
        got = B.fp4_norm_grad_pack8(dy, codes, scales, gamma, kind=kind, mean=f.mean, rstd=f.rstd, dres=dres)
        R.check(got.dh, dh, eh, "dh")
        R.check(got.dgamma, dg, eg, "dgamma")
        if layer:
            R.check(got.dbeta, db, eb, "dbeta")


@pytest.mark.parametrize("rows,cols", [(100, 512), (1000, 1024), (1100, 16416)])
def test_norm_grad_pack8_in_place(rows, cols):
    dev = device()
    announce(f"norm gradient of 8-bit rows in place {rows}x{cols}")
    h, dy, dres = (draw((rows, cols), i, BF).to(dev) for i in range(3))
    f = B.fp4_norm(h, save=True)
    codes, scales = B.fp4_pack8(h)
    args = dict(mean=f.mean, rstd=f.rstd, p=0.1, seed=2)
    want = B.fp4_norm_grad_pack8(dy, codes, scales, dres=dres, **args)
    ty, tr = dy.clone(), dres.clone()
    got = B.fp4_norm_grad_pack8(ty, codes, scales, dres=tr, dh=tr, dx=ty, **args)
    assert torch.equal(tr, want.dh) and torch.equal(ty, want.dx)
    assert torch.equal(got.dgamma, want.dgamma) and torch.equal(got.dbeta, want.dbeta)


def test_norm_gradient_against_differences():
    """With h as packing left it and its own statistics, dh and dgamma are the derivatives of sum(dy * norm(h)):
    central differences in binary64 along random directions, whose error is that of the binary32 gradient."""
    dev = device()
    announce("norm gradient of 8-bit rows against differences")
    rows, cols, eps = 6, 96, 1e-5
    codes, scales = B.fp4_pack8(draw((rows, cols), 1, F32, 2.0).to(dev))
    h = B.fp4_unpack8(codes, scales, out_dtype=F32)
    dy, gamma = draw((rows, cols), 2, F32).to(dev), (1 + draw((cols,), 3, F32, 0.2)).to(dev)
    f = B.fp4_norm(h, gamma, save=True)
    g = B.fp4_norm_grad_pack8(dy, codes, scales, gamma, mean=f.mean, rstd=f.rstd)

    def value(v, w):
        d = v - v.mean(1, keepdim=True)
        return float((dy.double().cpu() * d / (d.square().mean(1, keepdim=True) + eps).sqrt() * w).sum())

    v, w = h.double().cpu(), gamma.double().cpu()
    for i in range(4):
        dv, dw, t = draw((rows, cols), 10 + i, torch.float64), draw((cols,), 20 + i, torch.float64), 1e-4
        num = (value(v + t * dv, w) - value(v - t * dv, w)) / (2 * t)
        ana = float((g.dh.double().cpu() * dv).sum())
        assert abs(num - ana) < 1e-4 * float((g.dh.double().cpu() * dv).abs().sum())
        num = (value(v, w + t * dw) - value(v, w - t * dw)) / (2 * t)
        ana = float((g.dgamma.double().cpu() * dw).sum())
        assert abs(num - ana) < 1e-4 * float((g.dgamma.double().cpu() * dw).abs().sum())


@pytest.mark.parametrize("M,F,pair,pad", [(1, 16, 8, 0), (3, 64, 32, 8), (33, 4096, 32, 0), (7, 4096, 4096, 8),
                                          (65, 1040, 16, 0), (17, 11008, 32, 0)])
@pytest.mark.parametrize("want_h", [False, True])
def test_swiglu_grad_pack8(M, F, pair, pad, want_h):
    dev = device()
    announce(f"SwiGLU gradient of 8-bit rows {M}x{F} pair {pair} pad {pad} h {want_h}")
    c, dh = draw((M, 2 * F), 1, BF, 2.0), draw((M, F), 2, BF)
    codes, scales = B.fp4_pack8(c.to(dev))
    pd = Padded(M, F, BF, dev, pad, 0, dh)
    po, ph = Padded(M, 2 * F, BF, dev, pad, 0), Padded(M, F, BF, dev, pad, 0)
    dc, h = B.fp4_swiglu_grad_pack8(pd.view, codes, scales, pair=pair, dc=po.view, h=ph.view if want_h else None)
    values = B.fp4_unpack8(codes, scales)
    want = B.fp4_swiglu_grad_bf16(pd.view, values, pair=pair, want_h=want_h)
    same(dc, want[0], "dc")
    if want_h:
        same(h, want[1], "h")
    else:
        assert h is None
    assert po.untouched() and (ph.untouched() if want_h else bool((ph.buf == 777).all()))
    ref, _, err = R.swiglu_grad(dh, values.cpu(), pair)
    R.check(dc, ref, err, "dc")
    if want_h:
        t = pd.view  # h in the place of dh
        B.fp4_swiglu_grad_pack8(t, codes, scales, pair=pair, want_h=True, h=t)
        same(t, want[1], "h in place")


def test_swiglu_grad_pack8_nan():
    dev = device()
    announce("SwiGLU gradient of 8-bit rows with NaN")
    c = draw((4, 128), 1, BF)
    c[1, 3], c[2, 40] = math.inf, math.nan  # a gate, an up value
    dc, _ = B.fp4_swiglu_grad_pack8(torch.ones((4, 64), dtype=BF, device=dev), *B.fp4_pack8(c.to(dev)))
    bad = dc.isnan().cpu()
    want = torch.zeros_like(bad)
    want[1, 3] = want[1, 35] = want[2, 8] = True
    assert torch.equal(bad, want)


# ---------------------------------------------------------------- streams, graphs

def calls(dev, rows):
    cols = 1024
    x, r, dy = (draw((rows, cols), i, BF).to(dev) for i in range(3))
    c = draw((rows, 2 * cols), 3, BF).to(dev)
    gamma = (1 + draw((cols,), 4, F32, 0.2)).to(dev)

    def step(**s):
        c8 = B.fp4_pack8(c, **s)
        f = B.fp4_norm_pack8(x, gamma, residual=r, p=0.2, seed=4, save=True, mx=True, want_y=True, layout=B.LAYOUT_TILED, **s)
        h8 = B.fp4_pack8(f.h, **s)
        g = B.fp4_norm_grad_pack8(dy, *h8, gamma, mean=f.mean, rstd=f.rstd, p=0.2, seed=4, **s)
        return [*c8, *f, *h8, *g, B.fp4_unpack8(f.codes8, f.scales8, **s),
                *B.fp4_swiglu_grad_pack8(dy, *c8, want_h=True, **s)]

    return x, step


@pytest.mark.parametrize("rows", [100, 1200])
def test_named_stream(rows):
    dev = device()
    announce(f"8-bit rows on a stream of their own, {rows} rows")
    _, step = calls(dev, rows)
    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = step(stream=side)
    side.synchronize()
    for i, (a, b) in enumerate(zip(got, want)):
        assert torch.equal(a, b), f"output {i}"


@pytest.mark.parametrize("rows", [100, 1200])
def test_graph(rows):
    dev = device()
    announce(f"8-bit rows in a graph, {rows} rows")
    x, step = calls(dev, rows)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(3):
        x.copy_(draw((rows, 1024), 10 + k, BF).to(dev))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        assert all(torch.equal(a, b) for a, b in zip(got, step())), k
        torch.cuda.synchronize()

"""Products of few rows with FP4 weights on the GPU, against binary64 products
of the values that the operands stand for."""
import math

import numpy as np
import pytest
import torch

import oracle
from tests import pack8_ref as P
from tests import row_ref as R
from tests.gpu_common import B, announce, device
from tests.test_gpu_row_ops import Padded, draw

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
FORMATS = ["mx", "nv", "nv tile"]


def operand(fmt, n, k, seed, tiled, w=None):
    """(binary64 values [n, k], the call's tensors) of random FP4 weights, made by the oracle."""
    if w is None:
        g = torch.Generator().manual_seed(seed)
        w = torch.randn((n, k), generator=g) * torch.exp2(torch.randint(-3, 4, (n, k // 16), generator=g).float()
                                                          ).repeat_interleave(16, 1)
    x = w.to(BF)
    if fmt == "mx":
        c, s = oracle.quantize_mx(x.view(torch.int16).numpy().view(np.uint16))
        v, more = oracle.dequant_mx(c, s), []
        c, s = oracle.tile_mx(c, s) if tiled else (c, s)
    else:
        dom = oracle.NV_GLOBAL if fmt == "nv" else oracle.NV_TILE128
        c, s, ts = oracle.quantize_nv(x.view(torch.int16).numpy().view(np.uint16), domain=dom)
        v, more = oracle.dequant_nv(c, s, ts, dom), [torch.from_numpy(np.ascontiguousarray(ts, dtype=np.float32))]
        c, s = oracle.tile_nv(c, s) if tiled else (c, s)
    return v, [torch.from_numpy(np.ascontiguousarray(c)), torch.from_numpy(np.ascontiguousarray(s)), *more]


def matvec(fmt, x, w, tiled, **args):
    args["layout"] = B.LAYOUT_TILED if tiled else B.LAYOUT_LINEAR
    if fmt == "mx":
        return B.fp4_matvec_mx(x, *w, **args)
    return B.fp4_matvec_nv(x, *w, B.NV_GLOBAL if fmt == "nv" else B.NV_TILE128, **args)


def check(y, x, v, what, alpha=1.0):
    want = alpha * (x @ v.T)
    R.check(y, want, abs(alpha) * P.matvec_bound(x, v) + 2 * R.U * np.abs(want), what)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tiled", [False, True])
@pytest.mark.parametrize("m,n,k", [(1, 1, 128), (2, 15, 256), (1, 16, 128), (3, 17, 384), (16, 33, 256), (17, 100, 128),
                                   (5, 129, 2176), (32, 256, 1024), (33, 31, 512), (64, 200, 384), (1, 1000, 4096),
                                   (48, 130, 2048), (1, 300, 14336)])
def test_matvec(fmt, tiled, m, n, k):
    dev = device()
    announce(f"matvec {fmt} tiled {tiled} {m} x {n} x {k}")
    v, w = operand(fmt, n, k, m + n + k, tiled)
    w = [t.to(dev) for t in w]
    x = draw((m, k), n, BF)
    for out in (F32, BF):
        px, py = Padded(m, k, BF, dev, 8, 0, x), Padded(m, n, out, dev, 3, 1)
        got = matvec(fmt, px.view, w, tiled, n=n, y=py.view)
        check(got, x.double().numpy(), v, "y")
        assert py.untouched()
    made = matvec(fmt, x.to(dev), w, tiled, n=n, alpha=-0.375)
    assert made.dtype == F32
    check(made, x.double().numpy(), v, "y, alpha", -0.375)


@pytest.mark.parametrize("tiled", [False, True])
@pytest.mark.parametrize("m,n,k", [(1, 1, 128), (1, 100, 4096), (7, 50, 384), (16, 129, 256), (17, 33, 2176), (32, 256, 1024),
                                   (50, 31, 512), (64, 200, 384)])
def test_matvec_of_8_bit_rows(tiled, m, n, k):
    """As that of the rows unpacked, bit for bit, and against binary64."""
    dev = device()
    announce(f"matvec of 8-bit rows tiled {tiled} {m} x {n} x {k}")
    v, w = operand("mx", n, k, m + n + k, tiled)
    w = [t.to(dev) for t in w]
    x8 = B.fp4_pack8(draw((m, k), n, BF, 5.0).to(dev))
    layout = B.LAYOUT_TILED if tiled else B.LAYOUT_LINEAR
    for out in (F32, BF):
        py = Padded(m, n, out, dev, 3, 1)
        B.fp4_matvec_mx_pack8(*x8, *w, n=n, layout=layout, y=py.view)
        check(py.view, P.values(x8[0].cpu(), x8[1].cpu()), v, "y")
        assert py.untouched()
        same = B.fp4_matvec_mx(B.fp4_unpack8(*x8), *w, n=n, layout=layout, out_dtype=out)
        assert torch.equal(py.view, same)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tiled", [False, True])
@pytest.mark.parametrize("m,n", [(1, 16401), (20, 16384 + 31), (40, 16390), (3, 33000), (1, 70001)])
def test_many_weight_rows(fmt, tiled, m, n):
    dev = device()
    announce(f"matvec {fmt} tiled {tiled} {m} x {n} x 256")
    k = 256
    part, _ = operand(fmt, 512, k, 1, tiled)
    rows = torch.from_numpy(part).repeat(n // 512 + 1, 1)[:n] * torch.exp2(torch.arange(n) % 7 - 3.0)[:, None]
    v, w = operand(fmt, n, k, 1, tiled, rows.float())
    x = draw((m, k), 2, BF)
    got = matvec(fmt, x.to(dev), [t.to(dev) for t in w], tiled, n=n)
    check(got, x.double().numpy(), v, "y")
    if fmt == "mx":
        x8 = B.fp4_pack8(x.to(dev))
        got = B.fp4_matvec_mx_pack8(*x8, *[t.to(dev) for t in w], n=n, layout=B.LAYOUT_TILED if tiled else B.LAYOUT_LINEAR)
        check(got, P.values(x8[0].cpu(), x8[1].cpu()), v, "y of 8-bit rows")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tiled", [False, True])
@pytest.mark.parametrize("m,n", [(64, 28641), (49, 24570), (33, 20490), (32, 28641), (29, 24570), (16, 28641), (16, 24570)])
def test_many_rows_of_both(fmt, tiled, m, n):
    """Up to 112 rows of W to a wave."""
    dev = device()
    announce(f"matvec {fmt} tiled {tiled} {m} x {n} x 512")
    k = 512
    part, _ = operand(fmt, 256, k, 3, tiled)
    rows = torch.from_numpy(part).repeat(n // 256 + 1, 1)[:n] * torch.exp2(torch.arange(n) % 5 - 2.0)[:, None]
    v, w = operand(fmt, n, k, 3, tiled, rows.float())
    x = draw((m, k), 4, BF)
    got = matvec(fmt, x.to(dev), [t.to(dev) for t in w], tiled, n=n)
    check(got, x.double().numpy(), v, "y")


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("tiled", [False, True])
@pytest.mark.parametrize("each", [2, 3, 4, 5, 6, 7, 8])
def test_weight_rows_of_a_wave(fmt, tiled, each):
    """16 rows of W to a compute unit, twice that, and so on: every count of them to a wave."""
    dev = device()
    units, k = torch.cuda.get_device_properties(dev).multi_processor_count, 768 if each % 2 else 256
    n = 16 * units * each - 21
    announce(f"matvec {fmt} tiled {tiled} {n} x {k}")
    part, _ = operand(fmt, 256, k, each, tiled)
    rows = torch.from_numpy(part).repeat(n // 256 + 1, 1)[:n] * torch.exp2(torch.arange(n) % 3 - 1.0)[:, None]
    v, w = operand(fmt, n, k, each, tiled, rows.float())
    w = [t.to(dev) for t in w]
    for m in (4, 8, 16, 32, 64):
        x = draw((m, k), m, BF)
        check(matvec(fmt, x.to(dev), w, tiled, n=n), x.double().numpy(), v, f"y of {m} rows")


def test_weights_are_exact():
    """Each code times each MXFP4 scale that keeps it finite, and times each E4M3 scale, alone in its row."""
    dev = device()
    announce("matvec's weights, code by code")
    k = 128
    x = torch.zeros((1, k), dtype=BF)
    x[0, 37] = 1.0
    at = lambda c: (c << 4).astype(np.uint8)  # element 37 is a high nibble  # noqa: E731
    code, byte = (a.reshape(-1) for a in np.meshgrid(np.arange(16), np.arange(252), indexing="ij"))
    codes, scales = np.zeros((len(code), 64), np.uint8), np.zeros((len(code), 4), np.uint8)
    codes[:, 18], scales[:, 1] = at(code), byte
    got = B.fp4_matvec_mx(x.to(dev), torch.from_numpy(codes).to(dev), torch.from_numpy(scales).to(dev))
    want = oracle.dequant_mx(codes, scales)[:, 37]
    assert np.array_equal(got.cpu().double().numpy()[0], want)
    code, byte = (a.reshape(-1) for a in np.meshgrid(np.arange(16), np.arange(1, 127), indexing="ij"))
    codes, scales = np.zeros((len(code), 64), np.uint8), np.ones((len(code), 8), np.uint8)
    codes[:, 18], scales[:, 2] = at(code), byte
    got = B.fp4_matvec_nv(x.to(dev), torch.from_numpy(codes).to(dev), torch.from_numpy(scales).to(dev), torch.ones(1, device=dev))
    want = oracle.dequant_nv(codes, scales, np.ones(1, np.float32), oracle.NV_GLOBAL)[:, 37]
    assert np.array_equal(got.cpu().double().numpy()[0], want)


def test_8_bit_rows_of_all_scales():
    """Rows of blocks from the smallest to the largest scale: as their bf16 values, subnormal ones among them."""
    dev = device()
    announce("matvec of 8-bit rows of all scales")
    k = 128 * 62
    x8 = torch.randint(0, 127, (3, k), generator=torch.Generator().manual_seed(1), dtype=torch.uint8)
    s8 = (torch.arange(3 * k // 32) % 247).to(torch.uint8).reshape(3, k // 32)
    x8, s8 = x8.to(dev), s8.to(dev)
    codes = torch.zeros((k // 128, k // 2), dtype=torch.uint8)
    for i in range(k // 128):
        codes[i, 64 * i + 5] = 0x02  # a one at column 128 i + 10
        codes[i, 64 * i + 40] = 0x20  # and at 128 i + 81
    scales = torch.full((k // 128, k // 32), 127, dtype=torch.uint8)
    y = B.fp4_matvec_mx_pack8(x8, s8, codes.to(dev), scales.to(dev))
    v = B.fp4_unpack8(x8, s8).float().view(3, -1, 128)
    want = v[:, :, 10] + v[:, :, 81]
    assert torch.equal(y, want)
    read = v[:, :, [10, 81]]
    assert float(read[read > 0].min()) < 2.0 ** -126 and float(read.max()) > 2.0 ** 120


@pytest.mark.parametrize("fmt", FORMATS)
def test_nan_and_inf_stay_in_their_row(fmt):
    dev = device()
    announce(f"matvec {fmt} of NaN and Inf rows")
    m, n, k = 21, 70, 512
    v, w = operand(fmt, n, k, 3, True)
    w = [t.to(dev) for t in w]
    x = draw((m, k), 1, BF)
    clean = matvec(fmt, x.to(dev), w, True, n=n)
    x[2, 5], x[17, 300], x[20, 511] = math.nan, math.inf, -math.inf
    y = matvec(fmt, x.to(dev), w, True, n=n)
    assert bool(y[2].isnan().all()) and not bool(y[17].isfinite().any()) and not bool(y[20].isfinite().any())
    keep = [i for i in range(m) if i not in (2, 17, 20)]
    assert torch.equal(y[keep], clean[keep])
    if fmt == "mx":
        y = B.fp4_matvec_mx_pack8(*B.fp4_pack8(x.to(dev)), *w, n=n, layout=B.LAYOUT_TILED)
        assert bool(y[[2, 17, 20]].isnan().all()) and bool(y[keep].isfinite().all())


def test_empty():
    dev = device()
    announce("matvec of no rows, no weights, no columns")
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device=dev)  # noqa: E731
    x = torch.ones((3, 128), dtype=BF, device=dev)
    assert B.fp4_matvec_mx(x[:0], u8(5, 64), u8(5, 4)).shape == (0, 5)
    assert B.fp4_matvec_mx(x, u8(0, 64), u8(0, 4)).shape == (3, 0)
    for out in (F32, BF):
        y = torch.full((3, 37), 5.0, dtype=out, device=dev)
        B.fp4_matvec_mx(x[:, :0], u8(37, 0), u8(37, 0), y=y)
        assert bool((y == 0).all())
        y.fill_(5)
        B.fp4_matvec_nv(x[:, :0], u8(37, 0), u8(37, 0), torch.ones(1, device=dev), y=y)
        assert bool((y == 0).all())
        y.fill_(5)
        B.fp4_matvec_mx_pack8(u8(3, 0), u8(3, 0), u8(37, 0), u8(37, 0), y=y)
        assert bool((y == 0).all())


def test_too_many_rows():
    dev = device()
    announce("matvec of 65 rows")
    w = B.fp4_quantize_mx(torch.ones((40, 128), dtype=BF, device=dev))
    with pytest.raises(B.Fp4qError) as e:
        B.fp4_matvec_mx(torch.ones((65, 128), dtype=BF, device=dev), *w)
    assert e.value.status == B.EUNSUPPORTED


@pytest.mark.parametrize("tiled", [False, True])
def test_offsets_past_31_bits(tiled):
    """Codes past 2^31 bytes. (Against binary64: the order of the sums depends on the sizes, so that a small operand made
    of the far end's rows need not give the same bits.)"""
    dev = device()
    announce(f"matvec of 2.4 GB of codes, tiled {tiled}")
    k, n, last = 1 << 16, 73000 // 32 * 32, 64
    layout = B.LAYOUT_TILED if tiled else B.LAYOUT_LINEAR
    v, few = operand("mx", last, k, 1, tiled)
    codes = torch.zeros((n, k // 2), dtype=torch.uint8, device=dev)
    scales = torch.zeros((k // 128, n, 4) if tiled else (n, k // 32), dtype=torch.uint8, device=dev)
    codes[-last:] = few[0].to(dev)  # the tiled layout's groups of 32 rows are as long as 32 rows
    if tiled:
        scales[:, -last:] = few[1].to(dev)
    else:
        scales[-last:] = few[1].to(dev)
    x = draw((2, k), 2, BF)
    y = B.fp4_matvec_mx(x.to(dev), codes, scales, layout=layout)
    check(y[:, -last:], x.double().numpy(), v, "far rows")
    assert bool((y[:, :-last] == 0).all())


def test_same_bits_whatever_the_other_rows():
    """A token's result does not depend on which others it is batched with, within 16."""
    dev = device()
    announce("matvec batched and alone")
    _, w = operand("mx", 200, 2048, 4, True)
    w = [t.to(dev) for t in w]
    x = draw((16, 2048), 1, BF).to(dev)
    y = B.fp4_matvec_mx(x, *w, layout=B.LAYOUT_TILED, n=200)
    for i in range(16):
        assert torch.equal(B.fp4_matvec_mx(x[i:i + 1], *w, layout=B.LAYOUT_TILED, n=200), y[i:i + 1])


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n,k", [(200, 8192), (33, 14336), (2100, 1024), (4096, 512), (9000, 256)])
def test_same_bits_at_other_sizes(fmt, n, k):
    dev = device()
    tiled = n != 2100
    announce(f"matvec batched and alone {fmt} {n} x {k}")
    _, w = operand(fmt, n, k, 5, tiled)
    w = [t.to(dev) for t in w]
    x = draw((16, k), 6, BF).to(dev)
    y = matvec(fmt, x, w, tiled, n=n)
    for m in (1, 3, 4, 5, 8, 9, 13):
        assert torch.equal(matvec(fmt, x[16 - m:], w, tiled, n=n), y[16 - m:]), m


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("m", [9, 17, 24, 31, 33, 47, 49, 63])
def test_groups_of_rows(fmt, m):
    """Rows of x in several workgroups, the last of them short; rows and columns of W that end inside one."""
    dev = device()
    for n, k, tiled in ((130, 2048, True), (999, 512, False), (4100, 384, True), (4096, 256, False)):
        announce(f"matvec {fmt} groups of {m} rows {n} x {k}")
        v, w = operand(fmt, n, k, m + n, tiled)
        w = [t.to(dev) for t in w]
        x = draw((m, k), n, BF)
        px, py = Padded(m, k, BF, dev, 8, 0, x), Padded(m, n, BF, dev, 3, 1)
        check(matvec(fmt, px.view, w, tiled, n=n, y=py.view), x.double().numpy(), v, "y")
        assert py.untouched()
        if fmt == "mx":
            x8 = B.fp4_pack8(x.to(dev))
            got = B.fp4_matvec_mx_pack8(*x8, *w, n=n, layout=B.LAYOUT_TILED if tiled else B.LAYOUT_LINEAR)
            check(got, P.values(x8[0].cpu(), x8[1].cpu()), v, "y of 8-bit rows")


def test_streams_and_graph():
    dev = device()
    announce("matvec on other streams and in a graph")
    _, mx = operand("mx", 300, 1024, 1, True)
    _, nv = operand("nv tile", 300, 1024, 2, False)
    mx, nv = [t.to(dev) for t in mx], [t.to(dev) for t in nv]
    x = draw((4, 1024), 3, BF).to(dev)

    def step(**s):
        a = B.fp4_matvec_mx(x, *mx, layout=B.LAYOUT_TILED, n=300, **s)
        b = B.fp4_matvec_nv(x, *nv, B.NV_TILE128, **s)
        n = B.fp4_norm_pack8(x, kind=B.NORM_RMS, **s)
        return [a, b, B.fp4_matvec_mx_pack8(n.codes8, n.scales8, *mx, layout=B.LAYOUT_TILED, n=300, **s)]

    want = [t.clone() for t in step()]
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in range(3)]
    got = [step(stream=s) for s in sides]  # at once
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for k in range(3):
        x.copy_(draw((4, 1024), 10 + k, BF).to(dev))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        assert all(torch.equal(a, b) for a, b in zip(got, step())), k
        torch.cuda.synchronize()


def test_decoding_step():
    """One token (and a few) through a layer's MLP as a decoding step runs it: the residual's add and norm leave 8-bit
    rows, the gate/up product takes them, SwiGLU, the down product; against binary64 on the values each step had."""
    dev = device()
    announce("a decoding step's MLP")
    d, f = 512, 1024
    gu, wgu = operand("mx", 2 * f, d, 1, True, draw((2 * f, d), 1, F32, d ** -0.5))
    dn, wdn = operand("mx", d, f, 2, True, draw((d, f), 2, F32, f ** -0.5))
    wgu, wdn = [t.to(dev) for t in wgu], [t.to(dev) for t in wdn]
    gamma = (1 + draw((d,), 5, BF, 0.1)).to(dev)
    for m in (1, 5):
        x, r = draw((m, d), 3, BF).to(dev), draw((m, d), 4, BF).to(dev)
        n = B.fp4_norm_pack8(x, gamma, kind=B.NORM_RMS, residual=r)
        c = B.fp4_matvec_mx_pack8(n.codes8, n.scales8, *wgu, layout=B.LAYOUT_TILED, out_dtype=BF)
        h = B.fp4_swiglu_bf16(c, f)
        y = B.fp4_matvec_mx(h, *wdn, layout=B.LAYOUT_TILED, out_dtype=BF)
        check(c, P.values(n.codes8.cpu(), n.scales8.cpu()), gu, "c")
        check(y, h.double().cpu().numpy(), dn, "y")

"""Products of few rows with FP4 weights at the ends of what they take."""
import math

import numpy as np
import pytest
import torch

import oracle
from tests import pack8_ref as P
from tests.gpu_common import B, announce, device
from tests.test_gpu_matvec import check as matvec_check
from tests.test_gpu_row_ops import Padded, draw

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("alpha", [1.0, math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("m,n", [(1, 1), (5, 1031), (64, 37)])
def test_no_columns_give_zeros(alpha, m, n):
    """Whatever alpha is, as the GEMMs do, and nothing beside Y."""
    dev = device()
    announce(f"matvec {m} x {n} x 0, alpha {alpha}")
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device=dev)  # noqa: E731
    x = torch.ones((m, 0), dtype=BF, device=dev)
    for out in (F32, BF):
        for call in (lambda **a: B.fp4_matvec_mx(x, u8(n, 0), u8(n, 0), **a),
                     lambda **a: B.fp4_matvec_mx_pack8(u8(m, 0), u8(m, 0), u8(n, 0), u8(n, 0), **a),
                     lambda **a: B.fp4_matvec_nv(x, u8(n, 0), u8(n, 0), torch.ones(1, device=dev), **a)):
            py = Padded(m, n, out, dev, 3, 1)
            py.view.fill_(5.0)
            call(alpha=alpha, y=py.view)
            assert bool((py.view == 0).all()) and py.untouched()


def test_no_columns_of_many_rows():
    """More rows of W than 16 to a workgroup of 64 threads allow in one launch (nothing else bounds them at K = 0)."""
    dev = device()
    n = (1 << 30) + 77
    announce(f"matvec 1 x {n} x 0")
    y = torch.full((1, n), 5.0, dtype=BF, device=dev)
    none = torch.zeros((n, 0), dtype=torch.uint8, device=dev)
    B.fp4_matvec_mx(torch.ones((1, 0), dtype=BF, device=dev), none, none, y=y)
    assert not bool(y.any())
    del y, none
    torch.cuda.empty_cache()


def large_weights(n, k, seed):
    """(binary64 values, codes, scales in rows) of random codes whose blocks have scale bytes around 127, and every third
    in all but each fifth row one of 250 .. 254: weights up to 1.5 * 2^129."""
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (n, k // 2), generator=g, dtype=torch.uint8)
    scales = torch.randint(120, 134, (n, k // 32), generator=g, dtype=torch.uint8)
    top = torch.randint(250, 255, scales.shape, generator=g, dtype=torch.uint8)
    at = (torch.rand(scales.shape, generator=g) < 1 / 3) & (torch.arange(n) % 5 != 4)[:, None]
    scales = torch.where(at, top, scales)
    return oracle.dequant_mx(codes.numpy(), scales.numpy()).astype(np.float64), codes, scales


def largest(n, k, seed, tiled, dev):
    v, c, s = large_weights(n, k, seed)
    if tiled:
        c, s = (torch.from_numpy(np.ascontiguousarray(t)) for t in oracle.tile_mx(c.numpy(), s.numpy()))
    return v, [c.to(dev), s.to(dev)], dict(n=n, layout=B.LAYOUT_TILED if tiled else B.LAYOUT_LINEAR)


@pytest.mark.parametrize("tiled", [False, True])
@pytest.mark.parametrize("m,n,k", [(1, 70, 512), (5, 131, 384), (21, 70, 2048), (64, 200, 640), (1, 37, 14336), (12, 9000, 256)])
def test_weights_of_2_to_the_128_and_more(tiled, m, n, k):
    """Weights above bf16's largest value (E8M0 bytes 253 and 254): as the GEMM takes them, products that binary32
    holds come out within its sums' bound, and a zero in x stays a zero."""
    dev = device()
    announce(f"matvec of the largest MXFP4 weights, tiled {tiled} {m} x {n} x {k}")
    v, w, args = largest(n, k, m + n, tiled, dev)
    x = draw((m, k), 1, BF, 2.0 ** -20)
    x[1:][-1:] = 0
    for out in (F32, BF):
        py = Padded(m, n, out, dev, 3, 1)
        B.fp4_matvec_mx(x.to(dev), *w, y=py.view, **args)
        matvec_check(py.view, x.double().numpy(), v, "y")
        assert py.untouched() and not bool(py.view[1:][-1:].any())
        x8 = B.fp4_pack8(x.to(dev))
        y = B.fp4_matvec_mx_pack8(*x8, *w, out_dtype=out, alpha=0.25, **args)
        matvec_check(y, P.values(x8[0].cpu(), x8[1].cpu()), v, "y of 8-bit rows", 0.25)


@pytest.mark.parametrize("tiled", [False, True])
def test_largest_weights_by_themselves(tiled):
    """Each code at each of the largest scales, times 2^-20 (exact), 1 (2^128 and more are infinite in binary32) and 0."""
    dev = device()
    announce(f"matvec of the largest MXFP4 weights by themselves, tiled {tiled}")
    code, byte = (a.reshape(-1) for a in np.meshgrid(np.arange(16), np.arange(250, 256), indexing="ij"))
    codes, scales = np.zeros((len(code), 64), np.uint8), np.full((len(code), 4), 127, np.uint8)
    codes[:, 18], scales[:, 1] = (code << 4).astype(np.uint8), byte
    unit = np.where(byte == 255, np.nan, 2.0 ** (byte - 127.0))
    w = np.where(code < 8, 1, -1) * np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6])[code & 7] * unit
    if tiled:
        codes, scales = (np.ascontiguousarray(t) for t in oracle.tile_mx(codes, scales))
    x = torch.zeros((4, 128), dtype=BF)
    x[0, 37], x[1, 37], x[2, 5] = 2.0 ** -20, 1.0, 3.0
    y = B.fp4_matvec_mx(x.to(dev), torch.from_numpy(codes).to(dev), torch.from_numpy(scales).to(dev), n=len(code),
                        layout=B.LAYOUT_TILED if tiled else B.LAYOUT_LINEAR).cpu().numpy()
    assert np.array_equal(y[0].astype(np.float64), w * 2.0 ** -20, equal_nan=True)
    with np.errstate(over="ignore"):
        assert np.array_equal(y[1], w.astype(np.float32), equal_nan=True)
    assert np.array_equal(y[2:], np.where(byte == 255, np.nan, 0.0)[None].repeat(2, 0).astype(np.float32), equal_nan=True)


def test_largest_weights_batched_and_alone():
    """A row's bits are those of the row alone, and NaN and Inf stay in theirs."""
    dev = device()
    announce("matvec of the largest MXFP4 weights batched and alone")
    v, w, args = largest(9000, 1024, 3, True, dev)
    x = draw((16, 1024), 1, BF, 2.0 ** -20).to(dev)
    y = B.fp4_matvec_mx(x, *w, **args)
    assert bool(y.isfinite().all())
    for i in range(16):
        assert torch.equal(B.fp4_matvec_mx(x[i:i + 1], *w, **args), y[i:i + 1])
    bad = x.clone()
    bad[2, 5], bad[7, 1000] = math.nan, math.inf
    z = B.fp4_matvec_mx(bad, *w, **args)
    assert bool(z[2].isnan().all()) and not bool(z[7].isfinite().any())
    keep = [i for i in range(16) if i not in (2, 7)]
    assert torch.equal(z[keep], y[keep])

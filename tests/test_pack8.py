"""8-bit block-scaled rows and products of few rows with FP4 weights, without a
GPU: the library's refusals (before any HIP call; the addresses are never
dereferenced), the binding's checks, and the plain forms that the GPU's results
are held against."""
import math

import numpy as np
import pytest
import torch

from fp4_block_scaled_quantizer_amd import binding as B
from tests import made_up_addresses
from tests import pack8_ref as P
from tests.test_row_ops import RAN  # accepted (without a GPU: the launch fails)

A = [0x7F0000000000 + (i << 36) for i in range(14)]  # fake addresses far apart


@pytest.fixture(scope="module")
def L():
    return B.lib()


def test_reference_codes_are_torchs():
    r = np.random.RandomState(1)
    v = np.clip(np.concatenate([r.randn(20000) * 100, r.randn(20000) * 0.01, P.MIDDLE, -P.MIDDLE, P.E4M3]), -448, 448)
    v = v.astype(np.float32)
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(P.e4m3_codes(v.astype(np.float64)), want)
    assert np.array_equal(P.e4m3_values(want), torch.from_numpy(want).view(torch.float8_e4m3fn).double().numpy())


def test_reference_scales():
    x = torch.zeros((8, 32))
    x[1, 3] = 448.0
    x[2, 3] = -449.0
    x[3, 0], x[3, 1] = 2.0 ** -140, -(2.0 ** -149)
    x[4, 0] = torch.finfo(torch.float32).max
    x[5, 0], x[5, 1] = math.inf, 7.0
    x[6, 0], x[6, 31] = math.nan, 1.0
    x[7] = 1.75
    codes, scales = P.pack8(x)
    assert list(scales[:, 0] - 127.0) == [-127, 0, 1, -127, 119, -6, -8, -8]
    assert codes[5, 0] == 0x7F and codes[6, 0] & 0x7F == 0x7F
    v = P.values(codes, scales)
    assert v[1, 3] == 448 and v[2, 3] == -448 and v[4, 0] == 448 * 2.0 ** 119 and v[5, 1] == 7 and v[6, 31] == 1
    assert (v[7] == 1.75).all() and (v[3] == 0).all()


def test_pack8_error():
    """No element is off by more than half a step: 2^-4 of its value, or 2^(E - 10)."""
    g = torch.Generator().manual_seed(2)
    x = torch.randn((64, 256), generator=g) * torch.exp2(torch.randint(-60, 60, (64, 256), generator=g).float() / 8)
    codes, scales = P.pack8(x)
    unit = 2.0 ** np.repeat(scales.astype(int), 32, 1) / 2.0 ** 127
    err, v = np.abs(P.values(codes, scales) - x.double().numpy()), np.abs(x.double().numpy())
    assert (err <= np.maximum(v * 2.0 ** -4, unit * 2.0 ** -10)).all()


def test_pack8_refusals(L):
    def f(x=A[0], rows=4, cols=96, ld=100, t=1, codes=A[1], scales=A[2]):
        return [L.fp4_pack8(x, rows, cols, ld, t, codes, scales, None),
                L.fp4_unpack8(codes, scales, rows, cols, x, ld, t, None)]

    assert all(s in RAN for s in f() + f(t=0) + f(x=A[0] + 2) + f(scales=A[2] + 1) + f(ld=96))
    assert f(t=2) == [B.EINVAL] * 2
    assert f(cols=80) == [B.ESHAPE] * 2 and f(ld=95) == [B.ESHAPE] * 2 and f(rows=-1) == [B.ESHAPE] * 2
    assert f(rows=2 ** 31) == [B.ESHAPE] * 2 and f(ld=2 ** 31) == [B.ESHAPE] * 2
    assert f(rows=2 ** 20, cols=2 ** 15, ld=2 ** 15) == [B.ESHAPE] * 2  # 2^32 chunks
    for null in ("x", "codes", "scales"):
        assert f(**{null: None}) == [B.EINVAL] * 2
    assert f(x=A[0] + 1) == [B.EALIGN] * 2 and f(t=0, x=A[0] + 2) == [B.EALIGN] * 2
    assert f(codes=A[1] + 8) == [B.EALIGN] * 2
    assert f(codes=A[0]) == [B.EINVAL] * 2 and f(scales=A[0] + 8) == [B.EINVAL] * 2
    assert f(scales=A[1] + 16)[0] == B.EINVAL  # outputs overlap
    assert f(rows=0, x=None) == [B.OK] * 2 and f(cols=0, codes=None) == [B.OK] * 2


def test_norm_pack8_refusals(L):
    def f(x=A[0], rows=4, cols=128, ld=128, t=1, res=A[1], p=0.1, h=A[2], kind=0, g=A[3], b=A[4], y=A[5], mean=A[6],
          rstd=A[7], codes=A[8], scales=A[9], layout=0, c8=A[10], s8=A[11]):
        return L.fp4_norm_pack8(x, rows, cols, ld, t, res, 128, p, 1, 0, h, 128, kind, g, b, 0, 1e-5, y, 128, mean, rstd,
                                codes, scales, layout, c8, s8, None)

    assert f() in RAN and f(layout=1) in RAN and f(y=None, codes=None, scales=None) in RAN
    assert f(t=0, codes=None, scales=None) in RAN and f(s8=A[11] + 1) in RAN
    assert f(t=0) == B.EUNSUPPORTED                        # the MXFP4 operand of binary32 rows
    assert f(c8=None) == B.EINVAL and f(s8=None) == B.EINVAL and f(c8=None, s8=None) == B.EINVAL
    assert f(cols=112, codes=None, scales=None) == B.ESHAPE
    assert f(c8=A[10] + 8) == B.EALIGN
    for other in (A[0], A[1], A[2], A[3], A[5], A[6], A[8], A[9], A[11]):
        assert f(c8=other) == B.EINVAL
    assert f(s8=A[0] + 8) == B.EINVAL and f(s8=A[7]) == B.EINVAL
    assert f(kind=1) == B.EINVAL and f(kind=1, mean=None) in RAN and f(p=2.0) == B.EINVAL and f(x=None) == B.EINVAL
    assert f(rows=0, x=None, c8=None) == B.OK


def test_norm_grad_pack8_refusals(L):
    need = L.fp4q_norm_grad_workspace_bytes(4000, 128)

    def f(dy=A[0], rows=4000, cols=128, t=1, hc=A[1], hs=A[2], res=A[3], kind=0, g=A[4], mean=A[5], rstd=A[6], p=0.1,
          dh=A[7], dx=A[8], dg=A[9], db=A[10], ws=A[11], wb=need):
        return L.fp4_norm_grad_pack8(dy, rows, cols, 128, t, hc, hs, res, 128, kind, g, 0, mean, rstd, p, 1, 0, dh, 128,
                                     dx, 128, dg, db, ws, wb, None)

    assert f() in RAN and f(t=0) in RAN and f(dh=A[0]) in RAN and f(dh=A[3]) in RAN and f(hs=A[2] + 1) in RAN
    assert f(hc=None) == B.EINVAL and f(hs=None) == B.EINVAL and f(dy=None) == B.EINVAL and f(rstd=None) == B.EINVAL
    assert f(mean=None) == B.EINVAL and f(mean=None, kind=1) in RAN and f(wb=need - 1) == B.EINVAL
    assert f(cols=112) == B.ESHAPE and f(hc=A[1] + 4) == B.EALIGN
    assert f(dh=A[1]) == B.EINVAL and f(dx=A[2]) == B.EINVAL and f(dg=A[1]) == B.EINVAL and f(ws=A[2]) == B.EINVAL
    assert f(rows=0, dg=None, db=None, hc=None) == B.OK


def test_swiglu_grad_pack8_refusals(L):
    def f(dh=A[0], cc=A[1], cs=A[2], M=4, F=64, pair=32, dc=A[3], lddc=128, h=A[4]):
        return L.fp4_swiglu_grad_pack8(dh, 64, cc, cs, M, F, pair, dc, lddc, h, 64, None)

    assert f() in RAN and f(h=None) in RAN and f(h=A[0]) in RAN and f(cs=A[2] + 1) in RAN and f(F=48, pair=16) in RAN
    assert f(F=56, pair=8) == B.ESHAPE                     # 2F % 32
    assert f(F=60) == B.ESHAPE and f(pair=48) == B.ESHAPE and f(lddc=120) == B.ESHAPE and f(M=-1) == B.ESHAPE
    assert f(F=-16) == B.ESHAPE and f(F=2 ** 62) == B.ESHAPE
    assert f(cc=None) == B.EINVAL and f(cs=None) == B.EINVAL and f(dc=None) == B.EINVAL and f(dh=None) == B.EINVAL
    assert f(cc=A[1] + 8) == B.EALIGN
    assert f(dc=A[1]) == B.EINVAL and f(dc=A[2]) == B.EINVAL and f(h=A[1]) == B.EINVAL and f(h=A[2]) == B.EINVAL
    assert f(M=0, cc=None) == B.OK


def test_matvec_refusals(L):
    def mx(x=A[0], M=2, K=256, ld=256, c=A[1], s=A[2], N=100, layout=0, y=A[4], yt=1, ldy=100, **_):
        return L.fp4_matvec_mx(x, M, K, ld, c, s, N, 1.0, layout, y, yt, ldy, None)

    def mx8(x=A[0], xs=A[5], M=2, K=256, c=A[1], s=A[2], N=100, layout=0, y=A[4], yt=1, ldy=100, **_):
        return L.fp4_matvec_mx_pack8(x, xs, M, K, c, s, N, 1.0, layout, y, yt, ldy, None)

    def nv(x=A[0], M=2, K=256, ld=256, c=A[1], s=A[2], ts=A[3], dom=0, N=100, layout=0, y=A[4], yt=1, ldy=100, **_):
        return L.fp4_matvec_nv(x, M, K, ld, c, s, ts, dom, N, 1.0, layout, y, yt, ldy, None)

    for f in (mx, mx8, nv):
        assert f() in RAN and f(layout=1) in RAN and f(yt=0) in RAN and f(M=64) in RAN and f(ldy=104) in RAN
        assert f(layout=2) == B.EINVAL and f(yt=2) == B.EINVAL
        assert f(K=192) == B.ESHAPE and f(ldy=99) == B.ESHAPE and f(M=-1) == B.ESHAPE and f(N=-1) == B.ESHAPE
        assert f(N=2 ** 31, ldy=2 ** 31) == B.ESHAPE and f(N=2 ** 26, ldy=2 ** 26) == B.ESHAPE  # 2^32 bytes of codes and more
        assert f(M=65) == B.EUNSUPPORTED
        for null in ("x", "c", "s", "y"):
            assert f(**{null: None}) == B.EINVAL
        assert f(x=A[0] + 8) == B.EALIGN and f(c=A[1] + 8) == B.EALIGN and f(s=A[2] + 2) == B.EALIGN
        assert f(y=A[4] + 1) == B.EALIGN and f(yt=0, y=A[4] + 2) == B.EALIGN
        for other in (A[0], A[1], A[2]):
            assert f(y=other) == B.EINVAL
        assert f(M=0, x=None) == B.OK and f(N=0, x=None) == B.OK
        assert f(K=0, ld=0, x=None, c=None, s=None) in RAN  # zeros
    assert mx(ld=255) == B.ESHAPE and mx(ld=260) == B.EALIGN and nv(ld=260) == B.EALIGN
    assert mx8(xs=None) == B.EINVAL and mx8(y=A[5]) == B.EINVAL and mx8(xs=A[5] + 1) in RAN
    assert nv(ts=None) == B.EINVAL and nv(dom=2) == B.EINVAL and nv(dom=1) in RAN and nv(ts=A[3] + 2) == B.EALIGN
    assert nv(y=A[3]) == B.EINVAL
    assert nv(dom=1, y=A[3] + 4) == B.EINVAL and nv(dom=0, y=A[3] + 4) in RAN  # two tile scales, or one


def test_refusals_are_for_machines_without_a_gpu():
    for f in (test_pack8_refusals, test_norm_pack8_refusals, test_norm_grad_pack8_refusals, test_swiglu_grad_pack8_refusals,
              test_matvec_refusals):
        assert made_up_addresses.used_by(f)
    assert not made_up_addresses.used_by(test_binding_refusals)


def test_binding_refusals():
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    x, f, bf = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros(64), torch.bfloat16
    c, s, one = u8(4, 64), u8(4, 2), torch.ones(4)
    w, ws, v, vs, ts = u8(40, 64), u8(40, 4), u8(40, 64), u8(40, 8), torch.ones(1)
    x1 = torch.zeros((2, 128), dtype=bf)
    bad = [lambda: B.fp4_pack8(x.half()), lambda: B.fp4_pack8(x[0]), lambda: B.fp4_pack8(x[:, ::2]),
           lambda: B.fp4_pack8(x, codes=u8(4, 63)), lambda: B.fp4_pack8(x, scales=u8(4, 3)),
           lambda: B.fp4_pack8(x, codes=u8(8, 64)[::2]), lambda: B.fp4_pack8(x, codes=c.int()),
           lambda: B.fp4_unpack8(c, None), lambda: B.fp4_unpack8(c[0], s), lambda: B.fp4_unpack8(c, u8(4, 4)),
           lambda: B.fp4_unpack8(c.float(), s), lambda: B.fp4_unpack8(c, s, y=x[:2]),
           lambda: B.fp4_unpack8(c, s, y=x.half()), lambda: B.fp4_unpack8(c, s, out_dtype=torch.float16),
           lambda: B.fp4_unpack8(u8(4, 128)[:, ::2], s), lambda: B.fp4_unpack8(c, s, y=x[:1].expand(4, 64)),
           lambda: B.fp4_norm_pack8(x, f[:8]), lambda: B.fp4_norm_pack8(x, codes8=u8(4, 32)),
           lambda: B.fp4_norm_pack8(x, scales8=u8(4, 64)), lambda: B.fp4_norm_pack8(x[0], mx=True),
           lambda: B.fp4_norm_pack8(x, mx=True, codes=u8(4, 16)),
           lambda: B.fp4_norm_grad_pack8(x, c[:2], s, rstd=one), lambda: B.fp4_norm_grad_pack8(x, c, None, rstd=one),
           lambda: B.fp4_norm_grad_pack8(x, x, s, rstd=one), lambda: B.fp4_norm_grad_pack8(x, c, s, rstd=one[:3]),
           lambda: B.fp4_swiglu_grad_pack8(x, c, s), lambda: B.fp4_swiglu_grad_pack8(x, u8(4, 128), s),
           lambda: B.fp4_swiglu_grad_pack8(x.float(), u8(4, 128), u8(4, 4)),
           lambda: B.fp4_swiglu_grad_pack8(x, u8(4, 128), u8(4, 4), dc=x),
           lambda: B.fp4_matvec_mx(x1.float(), w, ws), lambda: B.fp4_matvec_mx(x1[0], w, ws),
           lambda: B.fp4_matvec_mx(x1, w[:, :32], ws), lambda: B.fp4_matvec_mx(x1, w, vs),
           lambda: B.fp4_matvec_mx(x1, w, ws, n=39), lambda: B.fp4_matvec_mx(x1, w, ws, layout=B.LAYOUT_TILED),
           lambda: B.fp4_matvec_mx(x1, u8(64, 64), u8(1, 64, 4), layout=B.LAYOUT_TILED, n=32),
           lambda: B.fp4_matvec_mx(x1, u8(64, 64), u8(64, 4), layout=B.LAYOUT_TILED),
           lambda: B.fp4_matvec_mx(x1, w, ws, y=torch.zeros((2, 41))),
           lambda: B.fp4_matvec_mx(x1, w, ws, y=torch.zeros((2, 40)).half()),
           lambda: B.fp4_matvec_mx(x1, w, ws, out_dtype=torch.float16),
           lambda: B.fp4_matvec_mx(x1, w.float(), ws), lambda: B.fp4_matvec_mx(x1, None, ws),
           lambda: B.fp4_matvec_mx_pack8(u8(2, 128), u8(2, 3), w, ws), lambda: B.fp4_matvec_mx_pack8(x1, u8(2, 4), w, ws),
           lambda: B.fp4_matvec_mx_pack8(u8(2, 128), None, w, ws),
           lambda: B.fp4_matvec_nv(x1, v, ws, ts), lambda: B.fp4_matvec_nv(x1, v, vs, None),
           lambda: B.fp4_matvec_nv(x1, v, vs, torch.ones(2)), lambda: B.fp4_matvec_nv(x1, v, vs, ts.double()),
           lambda: B.fp4_matvec_nv(torch.zeros((2, 256), dtype=bf), u8(200, 128), u8(200, 16), ts, B.NV_TILE128)]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError) as e:
            call()
        assert "current GPU" not in str(e.value), i
    for call in (lambda: B.fp4_pack8(x), lambda: B.fp4_unpack8(c, s), lambda: B.fp4_norm_pack8(x),
                 lambda: B.fp4_norm_grad_pack8(x, c, s, rstd=one, mean=one),
                 lambda: B.fp4_swiglu_grad_pack8(x, u8(4, 128), u8(4, 4)), lambda: B.fp4_matvec_mx(x1, w, ws),
                 lambda: B.fp4_matvec_mx(x1, u8(64, 64), u8(1, 64, 4), layout=B.LAYOUT_TILED, n=33),
                 lambda: B.fp4_matvec_mx_pack8(u8(2, 128), u8(2, 4), w, ws), lambda: B.fp4_matvec_nv(x1, v, vs, ts),
                 lambda: B.fp4_matvec_nv(torch.zeros((2, 256), dtype=bf), u8(200, 128), u8(200, 16), torch.ones((2, 2)),
                                         B.NV_TILE128)):
        with pytest.raises(ValueError, match="current GPU"):  # nothing wrong but the place
            call()


def test_binding_refuses_row_counts():
    """n has to be the operand's: a negative one is no request for all of them."""
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    x = torch.zeros((2, 128), dtype=torch.bfloat16)
    for n in (-1, -5, -40, 39, 41, 2**40, 2**62):
        for layout, ws in ((B.LAYOUT_LINEAR, u8(40, 4)), (B.LAYOUT_TILED, u8(1, 40, 4))):
            with pytest.raises(ValueError) as e:
                B.fp4_matvec_mx(x, u8(40, 64), ws, layout=layout, n=n)
            assert "current GPU" not in str(e.value), n
    with pytest.raises(ValueError, match="current GPU"):
        B.fp4_matvec_mx(x, u8(40, 64), u8(40, 4), n=40)

"""The row-wise operators' refusals (before any HIP call, so without a GPU;
the addresses are never dereferenced), the binding's checks, the dropout
counter against the oracle's Philox, and the long-context frequencies."""
import math

import numpy as np
import pytest
import torch

import oracle
from fp4_block_scaled_quantizer_amd import binding as B
from tests import row_ref as R

A = [0x7F0000000000 + (i << 36) for i in range(12)]  # fake addresses far apart
RAN = (B.OK, B.ELAUNCH)  # accepted (no GPU here: the launch fails)


@pytest.fixture(scope="module")
def L():
    return B.lib()


def test_dropout_refusals(L):
    def f(x=A[0], rows=4, cols=100, ld=100, t=1, res=A[1], ldr=100, p=0.1, y=A[2], ldy=100):
        return L.fp4_dropout(x, rows, cols, ld, t, res, ldr, p, 1, 0, y, ldy, None)

    assert f() in RAN and f(res=None, ldr=0) in RAN and f(x=A[0] + 2, ld=101) in RAN
    assert f(t=2) == B.EINVAL
    for p in (-0.1, 1.5, math.nan):
        assert f(p=p) == B.EINVAL
    assert f(x=None) == B.EINVAL and f(y=None) == B.EINVAL
    assert f(ld=99) == B.ESHAPE and f(ldy=99) == B.ESHAPE and f(ldr=99) == B.ESHAPE
    assert f(rows=-1) == B.ESHAPE and f(rows=2 ** 31) == B.ESHAPE and f(ld=2 ** 31) == B.ESHAPE
    assert f(rows=2 ** 20, cols=2 ** 15, ld=2 ** 15, ldr=2 ** 15, ldy=2 ** 15) == B.ESHAPE  # 2^32 chunks
    assert f(x=A[0] + 1) == B.EALIGN and f(t=0, y=A[2] + 2) == B.EALIGN
    assert f(y=A[0]) in RAN and f(y=A[1]) in RAN           # in place
    assert f(y=A[0], ldy=101) == B.EINVAL                  # another pitch
    assert f(y=A[0] + 16) == B.EINVAL
    assert f(rows=0, x=None, y=None) == B.OK and f(cols=0, x=None, y=None) == B.OK


def test_norm_refusals(L):
    def f(x=A[0], rows=4, cols=128, ld=128, t=1, res=A[1], ldr=128, p=0.1, h=A[2], ldh=128, kind=0, g=A[3], b=A[4], wt=0,
          eps=1e-5, y=A[5], ldy=128, mean=A[6], rstd=A[7], codes=A[8], scales=A[9], layout=0):
        return L.fp4_norm(x, rows, cols, ld, t, res, ldr, p, 1, 0, h, ldh, kind, g, b, wt, eps, y, ldy, mean, rstd, codes,
                          scales, layout, None)

    assert f() in RAN and f(layout=1) in RAN
    assert f(res=None, h=None, g=None, b=None, mean=None, rstd=None, codes=None, scales=None) in RAN
    assert f(y=None) in RAN
    assert f(y=None, codes=None, scales=None) == B.EINVAL  # no output
    assert f(codes=None) == B.EINVAL                       # scales without codes
    assert f(t=3) == B.EINVAL and f(wt=2) == B.EINVAL and f(kind=2) == B.EINVAL and f(layout=2) == B.EINVAL
    assert f(p=2.0) == B.EINVAL and f(eps=-1.0) == B.EINVAL and f(eps=math.nan) == B.EINVAL
    assert f(kind=1) == B.EINVAL and f(kind=1, mean=None) in RAN  # RMS has no mean
    assert f(x=None) == B.EINVAL
    assert f(ld=100) == B.ESHAPE and f(ldh=100) == B.ESHAPE and f(ldr=100) == B.ESHAPE and f(ldy=100) == B.ESHAPE
    assert f(cols=48, ld=128) == B.ESHAPE                  # K % 32 of the operand
    assert f(cols=96, layout=1) == B.ESHAPE                # K % 128, tiled
    assert f(t=0) == B.EUNSUPPORTED                        # codes of binary32 rows
    big = dict(ld=40000, ldr=40000, ldh=40000, ldy=40000)
    assert f(cols=32800, **big) == B.EUNSUPPORTED
    assert f(x=A[0] + 1) == B.EALIGN and f(g=A[3] + 2) == B.EALIGN and f(wt=1, g=A[3] + 2) in RAN
    assert f(codes=A[8] + 8) == B.EALIGN and f(layout=1, scales=A[9] + 4) == B.EALIGN and f(mean=A[6] + 2) == B.EALIGN
    assert f(h=A[1]) in RAN and f(y=A[0]) in RAN           # in place
    assert f(h=A[1], ldh=136) == B.EINVAL and f(y=A[2]) == B.EINVAL and f(y=A[3]) == B.EINVAL
    assert f(rstd=A[5]) == B.EINVAL and f(codes=A[0]) == B.EINVAL and f(scales=A[8]) == B.EINVAL
    assert f(rows=0, x=None) == B.OK


def test_norm_grad_refusals(L):
    need = L.fp4q_norm_grad_workspace_bytes(4000, 128)
    assert need > 0 and L.fp4q_norm_grad_workspace_bytes(0, 128) == 0
    assert L.fp4q_norm_grad_workspace_bytes(10 ** 6, 4096) == 256 * 2 * 4096 * 4

    def f(dy=A[0], rows=4000, cols=128, ld=128, t=1, h=A[1], ldh=128, res=A[2], ldr=128, kind=0, g=A[3], wt=0, mean=A[4],
          rstd=A[5], p=0.1, dh=A[6], ldd=128, dx=A[7], ldx=128, dg=A[8], db=A[9], ws=A[10], wb=need):
        return L.fp4_norm_grad(dy, rows, cols, ld, t, h, ldh, res, ldr, kind, g, wt, mean, rstd, p, 1, 0, dh, ldd, dx, ldx,
                               dg, db, ws, wb, None)

    assert f() in RAN and f(res=None, g=None, dx=None) in RAN and f(dh=None) in RAN
    assert f(dg=None, db=None, ws=None, wb=0) in RAN
    assert f(kind=1, mean=None, db=None) in RAN
    assert f(mean=None) == B.EINVAL and f(rstd=None) == B.EINVAL and f(dy=None) == B.EINVAL and f(h=None) == B.EINVAL
    assert f(dh=None, dx=None, dg=None, db=None) == B.EINVAL
    assert f(ws=None) == B.EINVAL and f(wb=need - 1) == B.EINVAL and f(ws=A[10] + 4) == B.EALIGN
    assert f(t=2) == B.EINVAL and f(kind=3) == B.EINVAL and f(p=math.nan) == B.EINVAL
    assert f(ld=127) == B.ESHAPE and f(ldx=127) == B.ESHAPE and f(rows=-1) == B.ESHAPE
    assert f(cols=32776, ld=40000, ldh=40000, ldr=40000, ldd=40000, ldx=40000) == B.EUNSUPPORTED
    assert f(dh=A[6] + 1) == B.EALIGN and f(dg=A[8] + 2) == B.EALIGN
    assert f(dh=A[0]) in RAN and f(dh=A[2]) in RAN and f(dx=A[1]) in RAN
    assert f(dh=A[0], ldd=130) == B.EINVAL and f(dx=A[6]) == B.EINVAL and f(dg=A[10]) == B.EINVAL and f(ws=A[1]) == B.EINVAL
    assert f(rows=0, dg=None, db=None) == B.OK


def test_swiglu_grad_refusals(L):
    def f(dh=A[0], ldd=64, c=A[1], M=16, F=64, ldc=128, pair=32, dc=A[2], lddc=128, h=A[3], ldh=64):
        return L.fp4_swiglu_grad_bf16(dh, ldd, c, M, F, ldc, pair, dc, lddc, h, ldh, None)

    assert f() in RAN and f(h=None, ldh=0) in RAN and f(dc=A[1]) in RAN and f(h=A[0]) in RAN
    assert f(F=60) == B.ESHAPE and f(pair=12) == B.ESHAPE and f(pair=48) == B.ESHAPE and f(ldc=120) == B.ESHAPE
    assert f(ldd=56) == B.ESHAPE and f(lddc=132) == B.ESHAPE and f(ldh=56) == B.ESHAPE and f(M=-1) == B.ESHAPE
    assert f(dh=None) == B.EINVAL and f(c=None) == B.EINVAL and f(dc=None) == B.EINVAL
    assert f(c=A[1] + 8) == B.EALIGN and f(h=A[3] + 2) == B.EALIGN
    assert f(dc=A[1], lddc=136) == B.EINVAL and f(dc=A[0]) == B.EINVAL and f(h=A[1]) == B.EINVAL
    assert f(M=0) == B.OK


def test_rotary_refusals(L):
    def f(x=A[0], n=4, heads=3, dim=64, xt=256, xh=64, t=1, pos=A[1], bits=64, fr=A[2], rot=64, style=0, inv=0, y=A[3],
          yt=192, yh=64):
        return L.fp4_rotary(x, n, heads, dim, xt, xh, t, pos, bits, fr, rot, style, inv, 1.0, y, yt, yh, None)

    assert f() in RAN and f(bits=32, style=1, inv=1, rot=32) in RAN and f(y=A[0], yt=256) in RAN
    assert f(t=2) == B.EINVAL and f(bits=16) == B.EINVAL and f(style=2) == B.EINVAL and f(inv=2) == B.EINVAL
    assert f(rot=0) == B.ESHAPE and f(rot=3) == B.ESHAPE and f(rot=66) == B.ESHAPE
    assert f(dim=1025, xh=1025, yh=1025) == B.ESHAPE and f(heads=65537) == B.ESHAPE
    assert f(xh=63) == B.ESHAPE and f(yt=191) == B.ESHAPE and f(n=-1) == B.ESHAPE
    assert f(x=None) == B.EINVAL and f(pos=None) == B.EINVAL and f(fr=None) == B.EINVAL and f(y=None) == B.EINVAL
    assert f(x=A[0] + 1) == B.EALIGN and f(pos=A[1] + 4) == B.EALIGN and f(fr=A[2] + 2) == B.EALIGN
    assert f(y=A[0]) == B.EINVAL and f(y=A[1]) == B.EINVAL and f(y=A[2]) == B.EINVAL  # y is x with another pitch; overlaps
    assert f(n=0, x=None) == B.OK and f(heads=0, x=None) == B.OK


def test_binding_refusals():
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    f = torch.zeros((32,))
    for call in (lambda: B.fp4_dropout(x.half(), 0.1, seed=1), lambda: B.fp4_dropout(x[0], 0.1, seed=1),
                 lambda: B.fp4_dropout(x[:, ::2], 0.1, seed=1), lambda: B.fp4_dropout(x, 0.1, seed=1, y=x.float()),
                 lambda: B.fp4_dropout(x, 0.1, seed=1, residual=x[:2]),
                 lambda: B.fp4_dropout(x[:1].expand(4, 64), 0.1, seed=1),
                 lambda: B.fp4_norm(x, f), lambda: B.fp4_norm(x, torch.zeros(64), torch.zeros(64).bfloat16()),
                 lambda: B.fp4_norm(x, torch.zeros(64).half()), lambda: B.fp4_norm(x, rstd=torch.zeros(3)),
                 lambda: B.fp4_norm(x, mx=True, codes=torch.zeros((4, 16), dtype=torch.uint8)),
                 lambda: B.fp4_norm_grad(x, x[:2], rstd=torch.zeros(4)),
                 lambda: B.fp4_norm_grad(x, x, rstd=torch.zeros(4).double()),
                 lambda: B.fp4_norm_grad(x, x, rstd=torch.zeros(4), dgamma=torch.zeros(63)),
                 lambda: B.fp4_swiglu_grad_bf16(x, x), lambda: B.fp4_swiglu_grad_bf16(x.float(), x),
                 lambda: B.fp4_swiglu_grad_bf16(x, torch.zeros((4, 128)).bfloat16(), dc=x),
                 lambda: B.fp4_rotary(x, torch.zeros(4, dtype=torch.int64), f),
                 lambda: B.fp4_rotary(x[:, None], torch.zeros(4), f),
                 lambda: B.fp4_rotary(x[:, None], torch.zeros(3, dtype=torch.int64), f),
                 lambda: B.fp4_rotary(x[:, None], torch.zeros(4, dtype=torch.int64), f.double()),
                 lambda: B.rotary_frequencies(63), lambda: B.rotary_frequencies(64, method="other"),
                 lambda: B.rotary_frequencies(64, method="linear", factor=0.5)):
        with pytest.raises(ValueError) as e:
            call()
        assert "current GPU" not in str(e.value)
    with pytest.raises(ValueError, match="current GPU"):  # nothing wrong but the place
        B.fp4_dropout(x, 0.1, seed=1)


def test_norm_grad_refusals_with_a_stream():
    x, one = torch.zeros((4, 64)), torch.ones(4)
    with pytest.raises(ValueError, match="2-D"):
        B.fp4_norm_grad(x[0], x[0], rstd=one, stream=object())
    with pytest.raises(ValueError, match="current GPU"):
        B.fp4_norm_grad(x, x, rstd=one, mean=one, stream=object())


def test_rotary_frequencies_refuses_an_empty_ramp():
    with pytest.raises(ValueError):
        B.rotary_frequencies(64, factor=4, method="turns", slow_turns=8, fast_turns=8)


def test_reference_draws_the_oracles_philox():
    k, r = np.meshgrid(np.arange(5), np.arange(7))
    w = R.philox_words(k, r, 9, 1, 0x123456789ABCDEF)
    for i in range(7):
        for j in range(5):
            want = oracle.philox4x32_10((j, i, 9, 1), (0x89ABCDEF, 0x01234567))
            assert [int(v[i, j]) for v in w] == [int(v) for v in want]


def test_rotary_frequencies():
    f, s = B.rotary_frequencies(64)
    assert s == 1.0 and f.dtype == torch.float32 and f[0] == 1 and f.shape == (32,)
    g, s = B.rotary_frequencies(64, factor=4, method="linear")
    assert s == 1.0 and torch.equal(g, f / 4)
    g, _ = B.rotary_frequencies(64, factor=4, method="base")
    assert g[0] == 1 and abs(float(g[-1] / f[-1]) - 0.25) < 1e-6
    g, s = B.rotary_frequencies(64, factor=4, method="turns", original_length=4096)
    turns = f.double() * 4096 / (2 * math.pi)
    assert torch.equal(g[turns > 32], f[turns > 32]) and torch.allclose(g[turns < 1], f[turns < 1] / 4)
    assert bool((g <= f).all()) and bool((g >= f / 4 * 0.999999).all()) and s == 1 + 0.1 * math.log(4)


def test_compiled_marshalling_is_required(monkeypatch):
    import sys
    monkeypatch.setitem(sys.modules, "fp4_block_scaled_quantizer_amd._row_calls", None)  # as if it were not built
    monkeypatch.delattr("fp4_block_scaled_quantizer_amd._row_calls", raising=False)
    monkeypatch.setattr(B, "_row_lib", None)
    with pytest.raises(FileNotFoundError, match="_row_calls"):
        B.fp4_dropout(torch.zeros((1, 8)), 0.5, seed=1)

"""Plain forms of 8-bit block-scaled rows and of products with FP4 weights, in
numpy's binary64 (test code)."""
import numpy as np

import oracle

# E4M3's finite magnitudes, codes 0 .. 0x7E: fields e, m stand for 2^(e - 7) (1 + m / 8), or m 2^-9 where e is 0
E4M3 = np.array([m * 2.0 ** -9 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7) for e in range(16) for m in range(8)][:127])
MIDDLE = (E4M3[1:] + E4M3[:-1]) / 2


def e4m3_codes(v):
    """E4M3 round to nearest even of finite v, magnitudes up to 448."""
    a = np.abs(v)
    assert (a <= 448).all()
    low = np.searchsorted(MIDDLE, a, side="left")  # a midpoint belongs to the lower of the two ...
    tie = (low < len(MIDDLE)) & (a == MIDDLE[np.minimum(low, len(MIDDLE) - 1)])
    code = np.where(tie & (low % 2 == 1), low + 1, low)  # ... unless that one is odd
    return (code + np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def e4m3_values(codes):
    c = np.asarray(codes).astype(int)
    v = np.append(E4M3, np.nan)[c & 127]
    return np.where(c >= 128, -v, v)


def scale_exponents(v):
    """E of each block of 32: the least integer with amax <= 448 2^E, by trying them."""
    b = np.abs(v.reshape(v.shape[0], -1, 32))
    amax = np.where(np.isfinite(b), b, 0).max(2)
    e = np.full(amax.shape, 119)
    for k in range(118, -128, -1):
        e = np.where(amax <= 448 * 2.0 ** k, k, e)
    return e


def pack8(x):
    """(codes, scales) of a 2-D torch tensor."""
    v = x.double().numpy()
    with np.errstate(all="ignore"):
        e = scale_exponents(v)
        unit = 2.0 ** np.repeat(e, 32, 1)
        fine = np.isfinite(v)
        y = np.clip(np.where(fine, v, 0) / unit, -448, 448)
        codes = np.where(fine, e4m3_codes(np.where(v < 0, -np.abs(y), y)), 0x7F + np.where(np.signbit(v), 128, 0))
    return codes.astype(np.uint8), (e + 127).astype(np.uint8)


def values(codes, scales):
    return e4m3_values(codes) * 2.0 ** (np.repeat(np.asarray(scales).astype(int), 32, 1) - 127.0)


def matvec_bound(x, w):
    """What binary32 sums may add to x w^T: an element's product passes through
    at most 32 sums inside an MFMA, one for each of a wave's MFMAs (32 columns
    each, at least a fourth of them in one wave where there are four steps or
    more) and one for each of up to 16 waves, alpha and the tensor scale add
    two, a tile's scale one for each step; matrix cores may cut where binary32
    rounds, which is twice as much."""
    k = x.shape[1]
    passes = 32 + max(k // 32 // 4, 4) + 16 + 2 + k // 128
    return 2 * passes * 2.0 ** -24 * (np.abs(x) @ np.abs(w).T)


def weights_mx(codes, scales):
    return oracle.dequant_mx(codes, scales).astype(np.float64)

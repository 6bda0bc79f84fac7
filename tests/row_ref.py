"""Plain binary64 forms of the row-wise operators, with the error that
binary32 evaluation may add (test code).

Error bounds count roundings of u = 2^-24: a sum that each lane forms over at
most 32 terms, joined over at most 64 lanes and 16 waves, passes any term
through fewer than 64 roundings, so it is off by at most 64 u times the sum
of magnitudes.  Results stored as bf16 add half a unit, 2^-9 of the value
(twice that covers a value pushed across a midpoint by the rest), results
stored as binary32 one u.
"""
import numpy as np
import torch

U = 2.0 ** -24
SUM = 64 * U


def store_error(want, dtype):
    rel = 2.0 ** -8 if dtype == torch.bfloat16 else 2 * U
    return np.abs(want) * rel + 2.0 ** -133


def philox_words(c0, c1, c2, c3, key):
    """Philox4x32-10 with Python integers on numpy object-free uint64 arrays."""
    m = np.uint64(0xFFFFFFFF)
    k0, k1 = key & 0xFFFFFFFF, key >> 32
    x = [np.asarray(v, dtype=np.uint64) for v in np.broadcast_arrays(c0, c1, c2, c3)]
    for r in range(10):
        a = x[0] * np.uint64(0xD2511F53)
        b = x[2] * np.uint64(0xCD9E8D57)
        x = [(b >> np.uint64(32)) ^ x[1] ^ np.uint64((k0 + r * 0x9E3779B9) & 0xFFFFFFFF), b & m,
             (a >> np.uint64(32)) ^ x[3] ^ np.uint64((k1 + r * 0xBB67AE85) & 0xFFFFFFFF), a & m]
    return x


def keep_mask(rows, cols, p, seed, stream_id=0):
    """(kept [rows, cols], scale as binary32)."""
    drop = int(np.rint(np.float64(np.float32(p)) * 65536))
    if drop == 0:
        return np.ones((rows, cols), bool), np.float32(1)
    k, r = np.meshgrid(np.arange(cols), np.arange(rows))
    w = np.stack(philox_words(k // 8, r, stream_id, 1, seed), 0)
    word = np.take_along_axis(w, ((k // 2) % 4)[None], 0)[0]
    r16 = np.where(k % 2 == 1, word >> np.uint64(16), word & np.uint64(0xFFFF))
    return r16 >= drop, np.float32(0 if drop == 65536 else 65536 / (65536 - drop))


def round_to(v32, dtype):
    return torch.from_numpy(np.ascontiguousarray(v32, dtype=np.float32)).to(dtype)


def dropout(x, residual, p, seed, stream_id=0):
    """Exactly the operator: binary32 product and sum, one rounding to x's type."""
    keep, scale = keep_mask(*x.shape, p, seed, stream_id)
    with np.errstate(invalid="ignore", over="ignore"):
        v = np.where(keep, x.float().numpy() * scale, np.float32(0)) if p > 0 else x.float().numpy()
        if residual is not None:
            v = residual.float().numpy() + v
    return round_to(v, x.dtype)


def norm(h, gamma, beta, layer, eps):
    """(y, mean, rstd, error bounds of the three) for rows h as stored."""
    v = h.double().numpy()
    n = v.shape[1]
    one = np.ones(n)
    g = one if gamma is None else gamma.double().numpy()
    b = 0 * one if beta is None else beta.double().numpy()
    mean = v.mean(1, keepdims=True) if layer else np.zeros((v.shape[0], 1))
    d = v - mean
    var = (d * d).mean(1, keepdims=True) + eps
    rstd = 1 / np.sqrt(var)
    y = d * rstd * g + b
    # the mean is off by SUM mean|h|; the deviations by that and u of themselves
    dmean = (SUM + 2 * U) * np.abs(v).mean(1, keepdims=True) if layer else np.zeros_like(mean)
    # d (var) / var <= SUM + 4 u + 2 |d| dmean / var (Cauchy: mean|d| <= sqrt(var)) + dmean^2 / var
    rel = 0.5 * (SUM + 8 * U + 2 * dmean * rstd + (dmean * rstd) ** 2) + 4 * U
    ey = np.abs(g) * rstd * (dmean + np.abs(d) * (rel + 6 * U)) + U * 2 * (np.abs(y) + np.abs(b))
    return y, mean, rstd, ey, dmean + U * np.abs(mean), rel * rstd


def norm_grad(dy, h, gamma, mean, rstd, layer, dres):
    """(dh, dgamma, dbeta, and their bounds before storing) from the statistics given."""
    e, v = dy.double().numpy(), h.double().numpy()
    rows, n = v.shape
    g = np.ones(n) if gamma is None else gamma.double().numpy()
    rs = rstd.double().numpy()[:, None]
    xh = (v - mean.double().numpy()[:, None] if layer else v) * rs
    gg = e * g
    c1 = (gg * xh).mean(1, keepdims=True)
    c2 = gg.mean(1, keepdims=True) if layer else np.zeros_like(c1)
    core = gg - c2 - xh * c1
    dh = core * rs
    ec1 = (SUM + 6 * U) * np.abs(gg * xh).mean(1, keepdims=True)
    ec2 = (SUM + 3 * U) * np.abs(gg).mean(1, keepdims=True)
    edh = rs * (ec2 + np.abs(xh) * ec1 + 6 * U * (np.abs(gg) + np.abs(c2) + np.abs(xh * c1)))
    if dres is not None:
        dh = dh + dres.double().numpy()
        edh = edh + U * 2 * np.abs(dh)
    # a weight's sum: rows / 256 terms and more in one lane, then at most 16
    # row groups, 16 parts of a slice and 16 slices
    k = (rows / 256 + 64 + 4) * U
    return dh, (e * xh).sum(0), e.sum(0), edh, k * np.abs(e * xh).sum(0), k * np.abs(e).sum(0)


def swiglu_grad(dh, c, pair):
    """(dc, h, bound of dc before storing) in binary64."""
    m, f = dh.shape
    cc = c.double().numpy()[:, :2 * f].reshape(m, f // pair, 2, pair)
    g, u, d = cc[:, :, 0], cc[:, :, 1], dh.double().numpy().reshape(m, f // pair, pair)
    with np.errstate(over="ignore"):
        s = 1 / (1 + np.exp(-g))
    act = g * s
    dg, du = d * u * (s + act * (1 - s)), d * act
    # sigma: the exponent's product with log2 e is off by |g| u relative to
    # e^-g, exp2, the sum and the reciprocal by 2 u each and a little
    rel = (1.5 * np.abs(g) + 10) * U
    eg = np.abs(d * u) * (rel * (s + 2 * np.abs(act) * (1 - s)) + 3 * U * (np.abs(act) + s)) + 2.0 ** -120
    eu = np.abs(du) * (rel + 2 * U) + 2.0 ** -120 * (1 + np.abs(d))
    return (np.stack([dg, du], 2).reshape(m, 2 * f), (act * u).reshape(m, f),
            np.stack([eg, eu], 2).reshape(m, 2 * f))


def rotary(x, positions, inv_freq, half_style, inverse, scale):
    """(y, bound before storing) in binary64."""
    v = x.double().numpy()
    nh = inv_freq.numel()
    # positions times a binary32 frequency is exact in binary64 up to 2^29
    t = positions.double().numpy()[:, None] * inv_freq.double().numpy()[None]
    c, s = np.cos(t)[:, None] * scale, np.sin(t)[:, None] * (-scale if inverse else scale)
    y = v.copy()
    ia = np.arange(nh) if half_style else 2 * np.arange(nh)
    ib = ia + nh if half_style else ia + 1
    a, b = v[..., ia], v[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    # sine and cosine: the fraction of a turn rounds to pi u of the angle, the
    # functions to 2 u, the scale to u; then three roundings of the sum
    e = np.zeros_like(v)
    e[..., ia] = e[..., ib] = (np.abs(a) + np.abs(b)) * abs(scale) * 10 * U + 2.0 ** -140
    return y, e


def check(got, want, err, what):
    got = got.detach().cpu()
    g = got.double().numpy()
    bound = err + store_error(want, got.dtype)
    bad = ~(np.abs(g - want) <= bound)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.size} out of bounds; first at {i}: {g[i]!r} for "
                             f"{want[i]!r}, bound {bound[i]:.3g}")

"""Measured cases of the row-wise operators between a transformer block's FP4
GEMMs: norm with residual and dropout, its gradient, dropout, rotary
positions, the gradient of SwiGLU.

`run` computes an operator in its plain form (elementary torch operations in
binary32) or, with `own` set, by the library's calls; `exact` is the same
operator from its definition in binary64.
"""
import math

import numpy as np
import torch

own = False

SEED = 0x1234567ABCDEF01  # the dropout key a training step carries
EPS = 1e-5
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}

# A micro-batch is 8192 tokens; model width 4096, fused QKV width 6144 (32
# query, 8 key and 8 value heads of 128), MLP width 14336.
MAX_ROW_WORK = 8192 * 4096
MAX_MLP_WORK = 8192 * 14336
MAX_ROTARY_WORK = 8192 * 40 * 128


def listed():
    return [
        # serving: the residual add and norm in front of a linear layer, for the one token being decoded
        dict(name="norm, one token", op="norm", rows=1, cols=4096, type="bf16", kind="rms", residual=True, p=0.0, pad=0),
        # training: dropout of a sub-block's output, residual add and layer norm over a micro-batch
        dict(name="norm, micro-batch", op="norm", rows=8192, cols=4096, type="bf16", kind="layer", residual=True,
             p=0.1, pad=0),
        # a width that no vector divides, unpadded binary32 rows
        dict(name="norm, odd binary32", op="norm", rows=1537, cols=5003, type="f32", kind="layer", residual=False,
             p=0.0, pad=0),
        # a short sequence's gradient in a narrow model
        dict(name="norm gradient, few rows", op="norm_grad", rows=96, cols=1024, type="bf16", kind="rms", dres=False,
             p=0.0, pad=0),
        # training: the gradient of "norm, micro-batch", the residual stream's gradient added, dropout undone
        dict(name="norm gradient, micro-batch", op="norm_grad", rows=8192, cols=4096, type="bf16", kind="layer",
             dres=True, p=0.1, pad=0),
        # wide binary32 rows, an odd number of them
        dict(name="norm gradient, wide", op="norm_grad", rows=2047, cols=14336, type="f32", kind="layer", dres=False,
             p=0.0, pad=0),
        # fine-tuning on a short prompt
        dict(name="dropout, short", op="dropout", rows=64, cols=4096, type="bf16", residual=False, p=0.1, pad=0),
        # dropout of the MLP's hidden activations of a micro-batch
        dict(name="dropout, micro-batch", op="dropout", rows=8192, cols=14336, type="bf16", residual=False, p=0.1,
             pad=0),
        # serving: queries and keys of 32 sequences' current tokens, inside the QKV GEMM's rows
        dict(name="rotary, decode", op="rotary", tokens=32, heads=40, dim=128, rot=128, style="half", inverse=False,
             row=6144, sequences=32),
        # training: the gradient's way back through a micro-batch of packed sequences
        dict(name="rotary, micro-batch", op="rotary", tokens=8192, heads=40, dim=128, rot=128, style="half",
             inverse=True, row=6144, sequences=7),
        # the MLP's gradient for a short sequence, gate and up interleaved as the fused GEMM writes them
        dict(name="swiglu gradient, short", op="swiglu_grad", rows=64, f=14336, pair=32, want_h=False),
        # the MLP's gradient for a micro-batch, the hidden activations recomputed for the weight's gradient
        dict(name="swiglu gradient, micro-batch", op="swiglu_grad", rows=8192, f=14336, pair=32, want_h=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_grad", "norm_grad", "dropout", "rotary", "swiglu_grad"])
    if op in ("norm", "norm_grad"):
        cols = _log(rng, 64, 16384)
        if rng.random() < 0.5:
            cols = cols // 32 * 32
        rows = _log(rng, 1, min(8192, MAX_ROW_WORK // (2 * cols)))
        return {"op": op, "rows": rows, "cols": cols, "type": rng.choice(["bf16", "bf16", "f32"]),
                "kind": rng.choice(["layer", "rms"]), "residual" if op == "norm" else "dres": rng.random() < 0.5,
                "p": rng.choice([0.0, 0.1, 0.25]), "pad": rng.choice([0, 0, 8, 24])}
    if op == "dropout":
        cols = _log(rng, 64, 28672)
        return dict(op=op, rows=_log(rng, 1, min(8192, MAX_MLP_WORK // (2 * cols))), cols=cols,
                    type=rng.choice(["bf16", "bf16", "f32"]), residual=rng.random() < 0.5,
                    p=rng.choice([0.05, 0.1, 0.5]), pad=rng.choice([0, 0, 8]))
    if op == "rotary":
        dim = rng.choice([64, 80, 96, 128, 192, 256])
        heads = _log(rng, 1, 64)
        tokens = _log(rng, 1, min(8192, MAX_ROTARY_WORK // (heads * dim)))
        return dict(op=op, tokens=tokens, heads=heads, dim=dim, rot=rng.choice([dim, dim, dim // 2]),
                    style=rng.choice(["half", "interleaved"]), inverse=rng.random() < 0.5,
                    row=dim * (heads + rng.choice([0, 2, 8])), sequences=min(tokens, rng.randrange(1, 9)))
    f = 32 * _log(rng, 2, 448)
    return dict(op=op, rows=_log(rng, 1, min(8192, MAX_MLP_WORK // f)), f=f, pair=rng.choice([32, f]),
                want_h=rng.random() < 0.5)


def _rows(g, rows, cols, pad, dtype, scale=1.0, outliers=False):
    """A [rows x cols] view with `pad` unused elements after each row: N(0, scale^2), with outliers one in a thousand
    entries fifty times as large, as activations have them."""
    x = torch.randn((rows, cols + pad), generator=g, device="cuda")
    if outliers:
        x = x * torch.where(torch.rand((rows, cols + pad), generator=g, device="cuda") < 1e-3, 50.0, 1.0)
    return (x * scale).to(dtype)[:, :cols]


def _room(rows, cols, dtype=torch.bfloat16):
    return torch.empty((rows, cols), dtype=dtype, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = dict(case, key=(SEED + seed) & (2 ** 63 - 1))
    if op in ("norm", "norm_grad", "dropout"):
        rows, cols, pad, dt = case["rows"], case["cols"], case["pad"], TYPES[case["type"]]
    if op in ("norm", "norm_grad"):
        s["gamma"] = (1 + 0.1 * torch.randn(cols, generator=g, device="cuda")).to(dt)
        s["beta"] = (0.1 * torch.randn(cols, generator=g, device="cuda")).to(dt) if case["kind"] == "layer" else None
    if op == "norm":
        s["x"] = _rows(g, rows, cols, pad, dt, outliers=True)
        s["res"] = _rows(g, rows, cols, pad, dt, scale=2.0) if case["residual"] else None
        s["y"] = _room(rows, cols, dt)
        s["h"] = _room(rows, cols, dt) if case["residual"] or case["p"] > 0 else None
        s["mean"] = _room(rows, 1, torch.float32)[:, 0] if case["kind"] == "layer" else None
        s["rstd"] = _room(rows, 1, torch.float32)[:, 0]
    elif op == "norm_grad":
        s["h"] = _rows(g, rows, cols, pad, dt, scale=2.0, outliers=True)
        s["dy"] = _rows(g, rows, cols, pad, dt, scale=1e-3)
        s["res"] = _rows(g, rows, cols, pad, dt, scale=1e-3) if case["dres"] else None
        h = s["h"].double()  # the statistics that the forward pass kept
        mean = h.mean(1, keepdim=True) if case["kind"] == "layer" else torch.zeros_like(h[:, :1])
        s["mean"] = mean[:, 0].float() if case["kind"] == "layer" else None
        s["rstd"] = ((h - mean).square().mean(1) + EPS).rsqrt().float()
        s["dh"], s["dx"] = _room(rows, cols, dt), _room(rows, cols, dt) if case["p"] > 0 else None
        s["dgamma"] = _room(1, cols, torch.float32)[0]
        s["dbeta"] = _room(1, cols, torch.float32)[0] if case["kind"] == "layer" else None
    elif op == "dropout":
        s["x"] = _rows(g, rows, cols, pad, dt)
        s["res"] = _rows(g, rows, cols, pad, dt) if case["residual"] else None
        s["y"] = _room(rows, cols, dt)
    elif op == "rotary":
        t, heads, dim = case["tokens"], case["heads"], case["dim"]
        qkv = torch.randn((t, case["row"]), generator=g, device="cuda").to(torch.bfloat16)
        s["x"] = qkv[:, :heads * dim].unflatten(1, (heads, dim))
        # packed sequences of equal share, each continuing from a prompt of its own length
        n = case["sequences"]
        start = torch.randint(0, 32768, (n,), generator=g, device="cuda")
        at = torch.arange(t, device="cuda")
        s["positions"] = start[at * n // t] + at - (at * n // t * t + n - 1) // n
        s["inv_freq"] = 500000.0 ** (-torch.arange(0, case["rot"], 2, device="cuda").float() / case["rot"])
        s["y"] = torch.empty((t, heads, dim), dtype=torch.bfloat16, device="cuda")
    else:
        m, f = case["rows"], case["f"]
        s["c"] = _rows(g, m, 2 * f, 0, torch.bfloat16, scale=1.5)
        s["dh"] = _rows(g, m, f, 0, torch.bfloat16, scale=1e-3)
        s["dc"] = _room(m, 2 * f)
        s["h"] = _room(m, f) if case["want_h"] else None
    return s


# ---------------------------------------------------------------- plain forms

def _philox(c0, c1, c2, c3, key):
    """Philox4x32-10 on int64 tensors that hold 32-bit words."""
    low = 0xFFFFFFFF
    k0, k1 = key & low, key >> 32
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = (p1 >> 32 & low) ^ c1 ^ k0, p1 & low, (p0 >> 32 & low) ^ c3 ^ k1, p0 & low
        k0, k1 = k0 + 0x9E3779B9 & low, k1 + 0xBB67AE85 & low
    return c0, c1, c2, c3


def _dropped(x, p, key):
    """x in binary32 with each element kept and scaled, or zero: element (r, k) draws 16 bits of the Philox words of
    counter (k / 8, r, 0, 1)."""
    if p == 0:
        return x.float()
    rows, cols = x.shape
    c8 = torch.arange((cols + 7) // 8, device=x.device)[None, :].expand(rows, -1)
    r = torch.arange(rows, device=x.device)[:, None].expand_as(c8)
    words = torch.stack(_philox(c8, r, torch.zeros_like(r), torch.ones_like(r), key), -1)
    r16 = torch.stack((words & 0xFFFF, words >> 16), -1).reshape(rows, -1)[:, :cols]
    drop = round(p * 65536)
    return torch.where(r16 >= drop, x.float() * (65536 / (65536 - drop)), 0.0)


def _plain_norm(s):
    x = _dropped(s["x"], s["p"], s["key"])
    h = (x if s["res"] is None else x + s["res"].float()).to(s["x"].dtype)
    v = h.float()
    mean = v.mean(1, keepdim=True) if s["kind"] == "layer" else torch.zeros_like(v[:, :1])
    d = v - mean
    rstd = (d.square().mean(1, keepdim=True) + EPS).rsqrt()
    y = d * rstd * s["gamma"].float()
    if s["beta"] is not None:
        y = y + s["beta"].float()
    out = {"y": y.to(h.dtype), "rstd": rstd[:, 0]}
    if s["h"] is not None:
        out["h"] = h
    if s["kind"] == "layer":
        out["mean"] = mean[:, 0]
    return out


def _plain_norm_grad(s):
    dy, h, rstd = s["dy"].float(), s["h"].float(), s["rstd"][:, None]
    layer = s["kind"] == "layer"
    xhat = (h - s["mean"][:, None] if layer else h) * rstd
    g = dy * s["gamma"].float()
    d = g - xhat * (g * xhat).mean(1, keepdim=True)
    if layer:
        d = d - g.mean(1, keepdim=True)
    dh = d * rstd
    if s["res"] is not None:
        dh = dh + s["res"].float()
    out = {"dh": dh.to(s["h"].dtype), "dgamma": (dy * xhat).sum(0)}
    if layer:
        out["dbeta"] = dy.sum(0)
    if s["p"] > 0:
        out["dx"] = _dropped(dh, s["p"], s["key"]).to(s["h"].dtype)
    return out


def _plain_dropout(s):
    y = _dropped(s["x"], s["p"], s["key"])
    return {"y": (y if s["res"] is None else y + s["res"].float()).to(s["x"].dtype)}


def _plain_rotary(s):
    x, rot = s["x"].float(), s["rot"]
    angle = s["positions"].float()[:, None, None] * s["inv_freq"]
    c, sn = angle.cos(), angle.sin()
    if s["inverse"]:
        sn = -sn
    a, b = (x[..., :rot // 2], x[..., rot // 2:rot]) if s["style"] == "half" else (x[..., 0:rot:2], x[..., 1:rot:2])
    ra, rb = a * c - b * sn, b * c + a * sn
    turned = torch.cat((ra, rb), -1) if s["style"] == "half" else torch.stack((ra, rb), -1).flatten(-2)
    return {"y": torch.cat((turned, x[..., rot:]), -1).to(s["x"].dtype)}


def _plain_swiglu_grad(s):
    m, f, pair = s["rows"], s["f"], s["pair"]
    c = s["c"].float().reshape(m, f // pair, 2, pair)
    g, u, dh = c[:, :, 0], c[:, :, 1], s["dh"].float().reshape(m, f // pair, pair)
    sig = 1 / (1 + torch.exp(-g))
    out = {"dc": torch.stack((dh * u * (sig * (1 + g * (1 - sig))), dh * (g * sig)), 2).to(s["c"].dtype).reshape(m, 2 * f)}
    if s["want_h"]:
        out["h"] = (g * sig * u).to(s["c"].dtype).reshape(m, f)
    return out


# ---------------------------------------------------------------- the library's calls

def _own_norm(s):
    from fp4_block_scaled_quantizer_amd import binding as B
    o = B.fp4_norm(s["x"], s["gamma"], s["beta"], kind=B.NORM_LAYER if s["kind"] == "layer" else B.NORM_RMS, eps=EPS,
                   residual=s["res"], p=s["p"], seed=s["key"], y=s["y"], h=s["h"], mean=s["mean"], rstd=s["rstd"])
    out = {"y": o.y, "rstd": o.rstd}
    if s["h"] is not None:
        out["h"] = o.h
    if s["kind"] == "layer":
        out["mean"] = o.mean
    return out


def _own_norm_grad(s):
    from fp4_block_scaled_quantizer_amd import binding as B
    o = B.fp4_norm_grad(s["dy"], s["h"], s["gamma"], kind=B.NORM_LAYER if s["kind"] == "layer" else B.NORM_RMS,
                        mean=s["mean"], rstd=s["rstd"], dres=s["res"], p=s["p"], seed=s["key"], dh=s["dh"],
                        dx=s["dx"], dgamma=s["dgamma"], dbeta=s["dbeta"])
    out = {"dh": o.dh, "dgamma": o.dgamma}
    if s["kind"] == "layer":
        out["dbeta"] = o.dbeta
    if s["p"] > 0:
        out["dx"] = o.dx
    return out


def _own_dropout(s):
    from fp4_block_scaled_quantizer_amd import binding as B
    return {"y": B.fp4_dropout(s["x"], s["p"], seed=s["key"], residual=s["res"], y=s["y"])}


def _own_rotary(s):
    from fp4_block_scaled_quantizer_amd import binding as B
    return {"y": B.fp4_rotary(s["x"], s["positions"], s["inv_freq"], inverse=s["inverse"], y=s["y"],
                              style=B.ROTARY_HALF if s["style"] == "half" else B.ROTARY_INTERLEAVED)}


def _own_swiglu_grad(s):
    from fp4_block_scaled_quantizer_amd import binding as B
    dc, h = B.fp4_swiglu_grad_bf16(s["dh"], s["c"], pair=s["pair"], dc=s["dc"], h=s["h"])
    return {"dc": dc, "h": h} if s["want_h"] else {"dc": dc}


PLAIN = dict(norm=_plain_norm, norm_grad=_plain_norm_grad, dropout=_plain_dropout, rotary=_plain_rotary,
             swiglu_grad=_plain_swiglu_grad)
OWN = dict(norm=_own_norm, norm_grad=_own_norm_grad, dropout=_own_dropout, rotary=_own_rotary,
           swiglu_grad=_own_swiglu_grad)


def run(state):
    return (OWN if own else PLAIN)[state["op"]](state)


def work(case):
    op = case["op"]
    if op in ("norm", "norm_grad", "dropout"):
        n, e = case["rows"] * case["cols"], 2 if case["type"] == "bf16" else 4
        layer = case.get("kind") == "layer"
    if op == "norm":  # x, [residual, h], y; gamma, [beta]; rstd, [mean]
        moved = n * e * (2 + case["residual"] + (case["residual"] or case["p"] > 0))
        return dict(bytes=moved + (1 + layer) * (case["cols"] * e + case["rows"] * 4), flops=10 * n)
    if op == "norm_grad":  # dy, h, [dres], dh, [dx]; gamma, dgamma, [dbeta]; rstd, [mean]
        moved = n * e * (3 + case["dres"] + (case["p"] > 0))
        return dict(bytes=moved + case["cols"] * (e + 4 + 4 * layer) + case["rows"] * 4 * (1 + layer), flops=15 * n)
    if op == "dropout":
        return dict(bytes=n * e * (2 + case["residual"]), flops=2 * n)
    if op == "rotary":
        n = case["tokens"] * case["heads"] * case["dim"]
        return dict(bytes=4 * n + 8 * case["tokens"] + 2 * case["rot"], flops=3 * n)
    n = case["rows"] * case["f"]
    return dict(bytes=n * (10 + 2 * case["want_h"]), flops=14 * n)


# ---------------------------------------------------------------- the definitions in 64 bits

def _words(counters, key):
    """Philox4x32-10 on the host: counters [n, 4] uint64, the four output words [n, 4]."""
    k = [key & 0xFFFFFFFF, key >> 32]
    c = [np.ascontiguousarray(counters[:, i]) for i in range(4)]
    mask, half = np.uint64(0xFFFFFFFF), np.uint64(32)
    for turn in range(10):
        left, right = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        key0 = np.uint64((k[0] + turn * 0x9E3779B9) % 2 ** 32)
        key1 = np.uint64((k[1] + turn * 0xBB67AE85) % 2 ** 32)
        c = [(right >> half) ^ c[1] ^ key0, right & mask, (left >> half) ^ c[3] ^ key1, left & mask]
    return np.stack(c, 1)


def _factor(rows, cols, p, key):
    """What dropout multiplies each element by, in binary64 on the GPU."""
    if p == 0:
        return 1.0
    groups = -(-cols // 8)
    n = np.zeros((rows * groups, 4), np.uint64)
    n[:, 0] = np.tile(np.arange(groups, dtype=np.uint64), rows)
    n[:, 1] = np.repeat(np.arange(rows, dtype=np.uint64), groups)
    n[:, 3] = 1
    bits = _words(n, key).astype(np.uint32).view(np.uint16).reshape(rows, groups * 8)[:, :cols]
    drop = int(round(p * 2 ** 16))
    kept = torch.from_numpy(np.ascontiguousarray(bits.astype(np.int32))).cuda() >= drop
    return kept.double() / (1 - drop / 2 ** 16)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    f64 = lambda t: t.to(torch.float64)  # noqa: E731
    if op == "dropout":
        y = f64(s["x"]).mul_(_factor(case["rows"], case["cols"], case["p"], s["key"]))
        return {"y": y if s["res"] is None else y.add_(s["res"])}
    if op == "norm":
        h = f64(s["x"]) * _factor(case["rows"], case["cols"], case["p"], s["key"])
        if s["res"] is not None:
            h = h + f64(s["res"])
        v = f64(h.to(s["x"].dtype))  # the statistics are those of h as it is kept
        n = case["cols"]
        mu = v.sum(1) / n if case["kind"] == "layer" else torch.zeros(case["rows"], dtype=torch.float64, device="cuda")
        inv = 1 / torch.sqrt(((v - mu[:, None]) ** 2).sum(1) / n + EPS)
        y = (v - mu[:, None]) * (inv[:, None] * f64(s["gamma"])[None])
        if s["beta"] is not None:
            y = y + f64(s["beta"])
        out = {"y": y, "rstd": inv}
        if s["h"] is not None:
            out["h"] = h
        if case["kind"] == "layer":
            out["mean"] = mu
        return out
    if op == "norm_grad":
        # with xhat and g = dy gamma the row's Jacobian is rstd (I - 1 1^T / n - xhat xhat^T / n)
        n, inv = case["cols"], f64(s["rstd"])
        xhat = f64(s["h"])
        if case["kind"] == "layer":
            xhat = xhat - f64(s["mean"])[:, None]
        xhat = xhat * inv[:, None]
        dy = f64(s["dy"])
        g = dy * f64(s["gamma"])
        along = (g * xhat).sum(1) / n
        level = g.sum(1) / n if case["kind"] == "layer" else torch.zeros_like(along)
        dh = inv[:, None] * (g - level[:, None] - xhat * along[:, None])
        if s["res"] is not None:
            dh = dh + f64(s["res"])
        out = {"dh": dh, "dgamma": (dy * xhat).sum(0)}
        if case["kind"] == "layer":
            out["dbeta"] = dy.sum(0)
        if case["p"] > 0:
            out["dx"] = dh * _factor(case["rows"], n, case["p"], s["key"])
        return out
    if op == "rotary":
        z = f64(s["x"])
        half = case["rot"] // 2
        turn = torch.exp(1j * (f64(s["positions"])[:, None] * f64(s["inv_freq"])[None])).conj() if case["inverse"] else \
            torch.exp(1j * (f64(s["positions"])[:, None] * f64(s["inv_freq"])[None]))
        y = z.clone()
        if case["style"] == "half":
            w = torch.complex(z[:, :, :half], z[:, :, half:2 * half]) * turn[:, None]
            y[:, :, :half], y[:, :, half:2 * half] = w.real, w.imag
        else:
            w = torch.complex(z[:, :, 0:2 * half:2], z[:, :, 1:2 * half:2]) * turn[:, None]
            y[:, :, 0:2 * half:2], y[:, :, 1:2 * half:2] = w.real, w.imag
        return {"y": y}
    # SwiGLU: h = u g sigma(g), d(g sigma)/dg = sigma + g sigma (1 - sigma)
    m, f, pair = case["rows"], case["f"], case["pair"]
    cols = torch.arange(f, device="cuda")
    at = cols // pair * 2 * pair + cols % pair
    g, u, dh = f64(s["c"][:, at]), f64(s["c"][:, at + pair]), f64(s["dh"])
    sig = torch.sigmoid(g)
    dc = torch.empty((m, 2 * f), dtype=torch.float64, device="cuda")
    dc[:, at + pair] = dh * g * sig
    dc[:, at] = dh * u * (sig + g * sig * (1 - sig))
    return {"dc": dc, "h": u * g * sig} if case["want_h"] else {"dc": dc}

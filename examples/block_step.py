"""Training steps of one transformer block whose linear layers run in MXFP4.

Everything between the GEMMs is the library's: the norms write the MXFP4
operand that the next GEMM loads, rotary positions are applied where the QKV
GEMM left the heads, dropout is drawn again instead of stored, and the MLP's
hidden activations are recomputed by SwiGLU's gradient. Attention itself is
written out in torch (binary32). With --keep8 what the backward pass reads of
the activations is kept in 8 bits. Synthetic data, random weights:

    python examples/block_step.py [--steps 8] [--tokens 512] [--width 1024] [--keep8]
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from fp4_block_scaled_quantizer_amd import binding as B  # noqa: E402

TILED = B.LAYOUT_TILED
SIGNS = 0x9E3779B9  # the fixed signs of the weight gradients' Hadamard transform


def linear(operand, w, m):
    """bf16 X W^T from X's MXFP4 operand."""
    return B.fp4_gemm_mx(*operand, *B.fp4_quantize_mx(w, layout=TILED), out_dtype=torch.bfloat16, layout=TILED, m=m,
                         n=w.shape[0])


class LinearGrad:
    """dY of a linear layer, read once into both operands it is needed as
    (stochastic rounding; Hadamard along tokens for the weight's gradient)."""

    def __init__(self, dy, seed):
        self.shape = dy.shape
        cr, sr, cc, sc = B.fp4_quantize_mx_dual(dy, round_rows=B.SR, stream_id_rows=0, hadamard_cols=True,
                                                sign_mask=SIGNS, round_cols=B.SR, stream_id_cols=1, seed=seed,
                                                layout=TILED)
        self.rows, self.cols = (cr, sr), (cc, sc)

    def x(self, w):
        wt = B.fp4_quantize_mx(w, axis=B.ALONG_COLS, layout=TILED)
        return B.fp4_gemm_mx(*self.rows, *wt, out_dtype=torch.bfloat16, layout=TILED, m=self.shape[0], n=w.shape[1])

    def w(self, x):
        xt = B.fp4_hadamard32_quantize(x, SIGNS, axis=B.ALONG_COLS, layout=TILED)
        return B.fp4_gemm_mx(*self.cols, *xt, alpha=1 / 32, layout=TILED, m=self.shape[1], n=x.shape[1])


def attention(q, k, v, sequence):
    """Causal attention inside each packed sequence, heads of q sharing those
    of k and v; [tokens, heads, dim] in binary32."""
    rep = q.shape[1] // k.shape[1]
    q, k, v = (t.transpose(0, 1).contiguous() for t in (q, k.repeat_interleave(rep, 1), v.repeat_interleave(rep, 1)))
    at = torch.arange(q.shape[1], device=q.device)
    hidden = (at[None] > at[:, None]) | (sequence[None] != sequence[:, None])
    s = torch.matmul(q, k.transpose(1, 2).contiguous()) / math.sqrt(q.shape[2])
    return torch.matmul(torch.softmax(s.masked_fill(hidden, float("-inf")), -1), v).transpose(0, 1)


class Rows:
    """Activations that the backward pass reads again: as they are."""

    def __init__(self, x):
        self.x = x

    def values(self):
        return self.x

    def norm_grad(self, dy, w, **args):
        return B.fp4_norm_grad(dy, self.x, w, kind=B.NORM_RMS, **args)

    def swiglu_grad(self, dh):
        return B.fp4_swiglu_grad_bf16(dh, self.x, want_h=True)


class Rows8:
    """The same in 8 bits, 33/64 of the bytes."""

    def __init__(self, x, packed=None):
        self.packed = B.fp4_pack8(x) if packed is None else packed

    def values(self):
        return B.fp4_unpack8(*self.packed)

    def norm_grad(self, dy, w, **args):
        return B.fp4_norm_grad_pack8(dy, *self.packed, w, kind=B.NORM_RMS, **args)

    def swiglu_grad(self, dh):
        return B.fp4_swiglu_grad_pack8(dh, *self.packed, want_h=True)


class Block:
    def __init__(self, width, heads, kv_heads, hidden, p, positions, sequence, seed=0, dim=128, keep8=False):
        g = torch.Generator().manual_seed(seed)
        self.heads, self.kv, self.dim, self.hidden, self.p = heads, kv_heads, dim, hidden, p
        self.positions, self.sequence, self.keep = positions, sequence, Rows8 if keep8 else Rows
        dev = positions.device

        def weight(n, k):
            return (torch.randn((n, k), generator=g) / math.sqrt(k)).to(dev)

        self.params = {"qkv": weight((heads + 2 * kv_heads) * dim, width), "o": weight(width, heads * dim),
                       "gate_up": B.pair_gate_up(weight(hidden, width), weight(hidden, width)),
                       "down": weight(width, hidden), "norm1": torch.ones(width, device=dev),
                       "norm2": torch.ones(width, device=dev)}
        self.freq, self.scale = B.rotary_frequencies(dim, 500000.0, device=dev)

    def turned(self, qkv):
        """The query and key heads inside the rows of a QKV matrix."""
        n = self.heads + self.kv
        return qkv[:, :n * self.dim].unflatten(1, (n, self.dim))

    def norm(self, x, w, **args):
        """The norm's outputs, and its result as the backward pass reads it."""
        args = dict(args, kind=B.NORM_RMS, save=True, mx=True, layout=TILED)
        if self.keep is Rows8:
            n = B.fp4_norm_pack8(x, w, **args)
            return n, Rows8(None, (n.codes8, n.scales8))
        n = B.fp4_norm(x, w, **args)
        return n, Rows(n.y)

    def forward(self, x, seed):
        w = {k: v.bfloat16() for k, v in self.params.items()}
        m, s = x.shape[0], {"x": self.keep(x), "seed": seed, "w": w}
        n1, s["y1"] = self.norm(x, w["norm1"])
        qkv = linear((n1.codes, n1.scales), w["qkv"], m)
        t = self.turned(qkv)
        B.fp4_rotary(t, self.positions, self.freq, scale=self.scale, y=t)
        heads = qkv.float().unflatten(1, (-1, self.dim)).split([self.heads, self.kv, self.kv], 1)
        s["qkv"] = [h.detach().requires_grad_() for h in heads]
        with torch.enable_grad():
            s["attention"] = attention(*s["qkv"], self.sequence)
        o = s["attention"].detach().flatten(1).bfloat16()
        a = linear(B.fp4_quantize_mx(o, layout=TILED), w["o"], m)
        n2, s["y2"] = self.norm(a, w["norm2"], residual=x, p=self.p, seed=seed, stream_id=0)
        c = linear((n2.codes, n2.scales), w["gate_up"], m)
        h = B.fp4_swiglu_bf16(c, self.hidden)
        d = linear(B.fp4_quantize_mx(h, layout=TILED), w["down"], m)
        s.update(o=self.keep(o), h2=self.keep(n2.h), c=self.keep(c), rstd1=n1.rstd, rstd2=n2.rstd)
        return B.fp4_dropout(d, self.p, seed=seed, stream_id=1, residual=n2.h), s

    def backward(self, dy, s):
        """(gradient of x, gradients of the parameters)."""
        w, seed, grad = s["w"], s["seed"], {}
        down = LinearGrad(B.fp4_dropout(dy, self.p, seed=seed, stream_id=1), seed + 1)
        dc, h = s["c"].swiglu_grad(down.x(w["down"]))
        grad["down"] = down.w(h)
        up = LinearGrad(dc, seed + 2)
        grad["gate_up"] = up.w(s["y2"].values())
        g = s["h2"].norm_grad(up.x(w["gate_up"]), w["norm2"], rstd=s["rstd2"], dres=dy, p=self.p, seed=seed, stream_id=0)
        grad["norm2"] = g.dgamma
        o = LinearGrad(g.dx if self.p > 0 else g.dh, seed + 3)
        grad["o"] = o.w(s["o"].values())
        s["attention"].backward(o.x(w["o"]).float().unflatten(1, (self.heads, self.dim)))
        dqkv = torch.cat([t.grad for t in s["qkv"]], 1).flatten(1).bfloat16()
        t = self.turned(dqkv)
        B.fp4_rotary(t, self.positions, self.freq, scale=self.scale, inverse=True, y=t)
        qkv = LinearGrad(dqkv, seed + 4)
        grad["qkv"] = qkv.w(s["y1"].values())
        g = s["x"].norm_grad(qkv.x(w["qkv"]), w["norm1"], rstd=s["rstd1"], dres=g.dh)
        grad["norm1"] = g.dgamma
        return g.dh, grad


def train(steps=8, tokens=512, width=1024, hidden=2816, heads=8, kv_heads=2, p=0.1, lr=0.5, seed=0, device="cuda",
          keep8=False):
    """Losses of `steps` steps that fit a fixed random target."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((tokens, width), generator=g).bfloat16().to(device)
    target = torch.randn((tokens, width), generator=g).to(device)
    at = torch.arange(tokens, device=device)
    cut = tokens * 5 // 8  # two packed sequences
    block = Block(width, heads, kv_heads, hidden, p, torch.where(at < cut, at, at - cut), (at >= cut).long(), seed,
                  keep8=keep8)
    losses = []
    for i in range(steps):
        y, saved = block.forward(x, 1000 * (seed + 1) + 10 * i)
        diff = y.float() - target
        losses.append(diff.square().mean())
        _, grad = block.backward((diff * (2 / width)).bfloat16(), saved)
        for name, v in grad.items():
            block.params[name] -= lr / tokens * v * (1.0 if v.dim() == 2 else 0.1)
    return [float(v) for v in losses]


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--width", type=int, default=1024)
    ap.add_argument("--keep8", action="store_true")
    a = ap.parse_args()
    for i, v in enumerate(train(a.steps, a.tokens, a.width, keep8=a.keep8)):
        print(f"step {i}: loss {v:.4f}")


if __name__ == "__main__":
    main()

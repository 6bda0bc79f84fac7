"""Training steps of one transformer block whose linear layers run in MXFP4.

Everything between the GEMMs is the library's: the norms write the MXFP4
operand that the next GEMM loads, rotary positions are applied where the QKV
GEMM left the heads, dropout is drawn again instead of stored, and the MLP's
hidden activations are recomputed by SwiGLU's gradient. Attention itself is
written out in torch (binary32). Synthetic data, random weights:

    python examples/block_step.py [--steps 8] [--tokens 512] [--width 1024]
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


class Block:
    def __init__(self, width, heads, kv_heads, hidden, p, positions, sequence, seed=0, dim=128):
        g = torch.Generator().manual_seed(seed)
        self.heads, self.kv, self.dim, self.hidden, self.p = heads, kv_heads, dim, hidden, p
        self.positions, self.sequence = positions, sequence
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

    def forward(self, x, seed):
        w = {k: v.bfloat16() for k, v in self.params.items()}
        m, s = x.shape[0], {"x": x, "seed": seed, "w": w}
        s["n1"] = B.fp4_norm(x, w["norm1"], kind=B.NORM_RMS, save=True, mx=True, layout=TILED)
        qkv = linear((s["n1"].codes, s["n1"].scales), w["qkv"], m)
        t = self.turned(qkv)
        B.fp4_rotary(t, self.positions, self.freq, scale=self.scale, y=t)
        heads = qkv.float().unflatten(1, (-1, self.dim)).split([self.heads, self.kv, self.kv], 1)
        s["qkv"] = [h.detach().requires_grad_() for h in heads]
        with torch.enable_grad():
            s["attention"] = attention(*s["qkv"], self.sequence)
        s["o"] = s["attention"].detach().flatten(1).bfloat16()
        a = linear(B.fp4_quantize_mx(s["o"], layout=TILED), w["o"], m)
        s["n2"] = B.fp4_norm(a, w["norm2"], kind=B.NORM_RMS, residual=x, p=self.p, seed=seed, stream_id=0, save=True,
                             mx=True, layout=TILED)
        s["c"] = linear((s["n2"].codes, s["n2"].scales), w["gate_up"], m)
        h = B.fp4_swiglu_bf16(s["c"], self.hidden)
        d = linear(B.fp4_quantize_mx(h, layout=TILED), w["down"], m)
        return B.fp4_dropout(d, self.p, seed=seed, stream_id=1, residual=s["n2"].h), s

    def backward(self, dy, s):
        """(gradient of x, gradients of the parameters)."""
        w, seed, grad = s["w"], s["seed"], {}
        down = LinearGrad(B.fp4_dropout(dy, self.p, seed=seed, stream_id=1), seed + 1)
        dc, h = B.fp4_swiglu_grad_bf16(down.x(w["down"]), s["c"], want_h=True)
        grad["down"] = down.w(h)
        up = LinearGrad(dc, seed + 2)
        grad["gate_up"] = up.w(s["n2"].y)
        g = B.fp4_norm_grad(up.x(w["gate_up"]), s["n2"].h, w["norm2"], kind=B.NORM_RMS, rstd=s["n2"].rstd, dres=dy,
                            p=self.p, seed=seed, stream_id=0)
        grad["norm2"] = g.dgamma
        o = LinearGrad(g.dx if self.p > 0 else g.dh, seed + 3)
        grad["o"] = o.w(s["o"])
        s["attention"].backward(o.x(w["o"]).float().unflatten(1, (self.heads, self.dim)))
        dqkv = torch.cat([t.grad for t in s["qkv"]], 1).flatten(1).bfloat16()
        t = self.turned(dqkv)
        B.fp4_rotary(t, self.positions, self.freq, scale=self.scale, inverse=True, y=t)
        qkv = LinearGrad(dqkv, seed + 4)
        grad["qkv"] = qkv.w(s["n1"].y)
        g = B.fp4_norm_grad(qkv.x(w["qkv"]), s["x"], w["norm1"], kind=B.NORM_RMS, rstd=s["n1"].rstd, dres=g.dh)
        grad["norm1"] = g.dgamma
        return g.dh, grad


def train(steps=8, tokens=512, width=1024, hidden=2816, heads=8, kv_heads=2, p=0.1, lr=0.5, seed=0, device="cuda"):
    """Losses of `steps` steps that fit a fixed random target."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((tokens, width), generator=g).bfloat16().to(device)
    target = torch.randn((tokens, width), generator=g).to(device)
    at = torch.arange(tokens, device=device)
    cut = tokens * 5 // 8  # two packed sequences
    block = Block(width, heads, kv_heads, hidden, p, torch.where(at < cut, at, at - cut), (at >= cut).long(), seed)
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
    a = ap.parse_args()
    for i, v in enumerate(train(a.steps, a.tokens, a.width)):
        print(f"step {i}: loss {v:.4f}")


if __name__ == "__main__":
    main()

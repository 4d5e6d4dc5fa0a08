"""Plain 64-bit references of the softmax-attention operators (torch on the CPU, one sequence and head
at a time) and the error bounds their GPU tests use.

The bounds count roundings.  u is half a step of the I/O type (eps / 2) and e = 2^-24 that of fp32.
A score is a sum of D fp32 products: it is off by at most (D + 8) e S with S = scale * sum |q k|, its
exponential by that much relative (twice: the score's own and the running maximum's) plus 4 e S for the
rounded argument; a sum over n keys adds n e.  Half-precision probabilities are rounded to the type
(u relative, and half of the smallest fp16 subnormal) before the second product, and the output once."""
from __future__ import annotations

import math

import torch

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
E32 = 2.0 ** -24


def half_step(kind: str) -> float:
    return torch.finfo(DT[kind]).eps / 2


def tiny_step(kind: str) -> float:
    """Half of the type's smallest subnormal: what a rounding can lose below the normal range."""
    f = torch.finfo(DT[kind])
    return f.tiny * f.eps / 2


def attention_ref(q, k, v, T, begin, kv_len, *, kind, prefix_k=None, prefix_v=None, scale=None):
    """q [N, H, D], k, v [rows, HK, D] (any strides, CPU); T, begin, kv_len per sequence.  Returns
    (out, lse, out bound, lse bound) in 64 bits."""
    N, H, D = q.shape
    HK = k.shape[1]
    G = H // HK
    scale = 1 / math.sqrt(D) if scale is None else scale
    u, sub = half_step(kind), tiny_step(kind)
    out = torch.zeros(q.shape, dtype=torch.float64)
    lse = torch.full((N, H), -math.inf, dtype=torch.float64)
    out_tol, lse_tol = torch.zeros_like(out), torch.zeros_like(lse)
    start = 0
    for b, t in enumerate(T):
        for h in range(H if t else 0):
            hk = h // G
            kk, vv = (x[begin[b]:begin[b] + kv_len[b], hk].double() for x in (k, v))
            P = 0
            if prefix_k is not None:
                P = prefix_k.shape[0]
                kk, vv = torch.cat((prefix_k[:, hk].double(), kk)), torch.cat((prefix_v[:, hk].double(), vv))
            qq = q[start:start + t, h].double()
            j = torch.arange(len(kk))
            hidden = (j >= P) & (j - P > (kv_len[b] - t + torch.arange(t))[:, None])  # the prefix is seen by all
            s = (qq @ kk.T * scale).masked_fill(hidden, -math.inf)
            S = (qq.abs() @ kk.abs().T * abs(scale)).masked_fill(hidden, 0.0)
            if len(kk) == 0:
                continue
            S = S.amax(-1)
            n = (~hidden).sum(-1)
            top = s.amax(-1, keepdim=True)
            p = torch.exp(s - torch.where(top == -math.inf, 0.0, top))
            l = p.sum(-1, keepdim=True)
            some = l > 0
            p = p / torch.where(some, l, 1.0)
            # rows a token does not see take no part, whatever they hold
            vis = torch.where(hidden.all(0)[:, None], 0.0, vv)
            if torch.isfinite(vis).all():
                o, o_abs = p @ vis, p @ vis.abs()
                v_sum = (~hidden).double() @ vis.abs()
            else:
                pick = [torch.where(hidden[i][:, None], 0.0, vv) for i in range(t)]
                o = torch.stack([p[i] @ x for i, x in enumerate(pick)])
                o_abs = torch.stack([p[i] @ x.abs() for i, x in enumerate(pick)])
                v_sum = torch.stack([x.abs().sum(0) for x in pick])
            out[start:start + t, h] = o
            lse[start:start + t, h] = (top + l.log()).squeeze(-1)
            gamma = ((2 * (D + 8) + 4) * S + 2 * n + 32) * E32
            rel = (gamma + (0.0 if kind == "f32" else 2 * u))[:, None]
            # P below fp16's normal range: half a subnormal step against a sum of at least l >= 1
            flat = 0.0 if kind == "f32" else sub * v_sum / torch.where(some, l, 1.0)
            out_tol[start:start + t, h] = rel * o_abs + u * o.abs() + flat + sub
            lse_tol[start:start + t, h] = ((D + 12) * S + n + 32) * E32 + 8 * E32 * top.squeeze(-1).abs().clamp(max=1e30)
        start += t
    return out, lse, out_tol, lse_tol


def rope_ref(x, weight, pos, inv_freq, *, eps, interleaved, kind):
    """Norm and rotation of x [T, heads, D] at the positions pos (CPU): (value, bound) in 64 bits.

    The norm's sum (a tree over at most 8 terms a lane and 6 levels), root, quotient and two products
    are off by at most 16 e relative; the fraction of a turn is rounded to fp32 (2 pi 2^-26 of angle) and
    its sine and cosine to 2 e of 1, two products and a sum add 3 e: 24 e of |lo| + |hi| covers both."""
    y = x.double()
    y = y / torch.sqrt(y.square().mean(-1, keepdim=True) + eps)
    if weight is not None:
        y = y * weight.double()
    mag = y.abs()
    half = len(inv_freq)
    angle = pos.double()[:, None] * inv_freq.double()
    cos, sin = angle.cos()[:, None], angle.sin()[:, None]
    lo, hi = (slice(0, 2 * half, 2), slice(1, 2 * half, 2)) if interleaved else (slice(0, half), slice(half, 2 * half))
    z = y.clone()
    z[..., lo] = y[..., lo] * cos - y[..., hi] * sin
    z[..., hi] = y[..., lo] * sin + y[..., hi] * cos
    both = mag[..., lo] + mag[..., hi]
    mag[..., lo] = both
    mag[..., hi] = both
    return z, 24 * E32 * mag + half_step(kind) * z.abs() + tiny_step(kind)


def assert_within(got, ref, tol, what):
    """|got - ref| <= tol element by element; infinities have to be equal."""
    got = got.double().cpu()
    same = (got == ref) & torch.isinf(ref)
    d = (got - ref).abs()
    bad = ~(same | (d <= tol))
    worst = (d / tol.clamp(min=1e-300)).masked_fill(same, 0.0).max().item() if d.numel() else 0.0
    print(f"[err] {what}: largest error {worst:.3f} of its bound", flush=True)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} out of bounds, worst {worst:.3g} of the bound at {bad.nonzero()[0].tolist()}"


def layout(lengths, gap=3, order=None):
    """Cache runs for the (T, n) lengths, in the given order, `gap` unused rows before and after each:
    (begin per sequence, rows)."""
    begin, rows = [0] * len(lengths), gap
    for b in order if order is not None else range(len(lengths)):
        begin[b] = rows
        rows += lengths[b][1] + gap
    return begin, rows

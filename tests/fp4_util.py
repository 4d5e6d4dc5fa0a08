"""Plain 64-bit references of the 4-bit cache and the block's norms (torch on the CPU), with the error bounds of their GPU
tests.  e = 2^-24 is half a step of fp32, u that of the I/O type; the sums of these kernels add at most 64 terms in a
thread, six levels in a wave and 16 waves, so a sum of positive terms is off by at most 86 e relative and the inverse of
its root by 43 + 4 e."""
from __future__ import annotations

import torch

from attn_util import DT, E32, half_step, tiny_step

VALUES = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
LOWEST, HIGHEST = {"f32": -126, "bf16": -126, "f16": -23}, {"f32": 125, "bf16": 125, "f16": 13}
SUM = 86


def encode(x, kind):
    """(codes [..., D/2], scales [..., D/32]) uint8 of x [..., D]: the nearest of the 15 values by distance, ties to the
    even code, with the least power of two whose 6-fold holds the block."""
    y = x.double().unflatten(-1, (-1, 32))
    top = y.abs().amax(-1)
    bad = ~torch.isfinite(y).all(-1)
    y, top = torch.where(bad[..., None], 0.0, y), torch.where(bad, 0.0, top)
    e = torch.full(top.shape, LOWEST[kind], dtype=torch.int64)
    for _ in range(HIGHEST[kind] - LOWEST[kind]):
        more = (top > 6 * 2.0 ** e.double()) & (e < HIGHEST[kind])
        if not more.any():
            break
        e = e + more
    size = (y * 2.0 ** -e.double()[..., None]).abs()
    far = (size[..., None] - VALUES).abs()
    code = far.argmin(-1)  # the lower of two equally near codes
    up = (code + 1).clamp(max=7)
    tie = (far.gather(-1, up[..., None]) == far.gather(-1, code[..., None])).squeeze(-1) & (code % 2 == 1)
    code = torch.where(tie, up, code) | (torch.signbit(y).long() << 3)
    code = torch.where(bad[..., None], 0, code).flatten(-2)
    return (code[..., 0::2] | code[..., 1::2] << 4).byte(), torch.where(bad, 255, e + 127).byte()


def decode(codes, scales):
    """The values in 64 bits."""
    c = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).long()
    y = torch.where(c >= 8, -VALUES[c & 7], VALUES[c & 7])
    s = torch.where(scales == 255, float("nan"), 2.0 ** (scales.double() - 127))
    return (y.unflatten(-1, (-1, 32)) * s[..., None]).flatten(-2)


def strided(x, layout):
    """A copy of x [rows, heads, w] on the device: "rows" contiguous, "heads" heads outermost, "wide" parts of wider rows."""
    x = x.to("cuda")
    if layout == "heads":
        return x.permute(1, 0, 2).contiguous().permute(1, 0, 2)
    if layout == "wide":
        rows, heads, w = x.shape
        room = torch.full((rows, heads + 2, w), 255 if x.dtype == torch.uint8 else float("nan"), dtype=x.dtype, device="cuda")
        room[:, 1:1 + heads] = x
        return room[:, 1:1 + heads]
    return x.contiguous()


def residual_ref(x, residual, weight, post_weight, scale, channel_scale, eps, kind, stream):
    """(out, residual_out, bound, bound) in 64 bits."""
    t = x.double()
    rel = 4.0  # products with the scales
    if post_weight is not None:
        t = t / torch.sqrt(t.square().mean(-1, keepdim=True) + eps) * post_weight.double()
        rel += SUM / 2 + 6
    t = t * scale
    if channel_scale is not None:
        t = t * channel_scale.double()
    h = t if residual is None else residual.double() + t
    dh = rel * E32 * t.abs() + E32 * h.abs()
    root = torch.sqrt(h.square().mean(-1, keepdim=True) + eps)
    y = h / root
    moved = torch.sqrt(dh.square().mean(-1, keepdim=True)) / root
    w = 1.0 if weight is None else weight.double()
    y = y * w
    tol = dh / root * abs(w) + y.abs() * ((SUM / 2 + 8) * E32 + moved + half_step(kind)) + tiny_step(kind)
    return y, h, 1.01 * tol, 1.01 * (dh + half_step(stream) * h.abs()) + tiny_step(stream)


def gated_ref(x, gate, weight, eps, activation, gate_first, norm, kind):
    """(out, bound) in 64 bits.  The exponential's argument is off by two roundings of |gate|, itself, the sum and the
    reciprocal by two each; past 2^127 the exponential is infinite, which moves the gate by less than 2^-126."""
    x, g = x.double(), gate.double()
    act = torch.sigmoid(g)
    far = 2.0 ** -126 * torch.ones_like(g)
    if activation == "silu":
        act, far = g * act, far * g.abs()
    rel_act = (2 * g.abs() + 9) * E32
    y = x * act if gate_first else x
    dy = y.abs() * (rel_act + E32) + far * x.abs() if gate_first else torch.zeros_like(y)
    w = 1.0 if weight is None else weight.double()
    if norm:
        root = torch.sqrt(y.square().mean(-1, keepdim=True) + eps)
        moved = torch.sqrt(dy.square().mean(-1, keepdim=True)) / root
        dy = (dy / root + (y / root).abs() * ((SUM / 2 + 8) * E32 + moved)) * abs(w)
        y = y / root * w
    if not gate_first:
        dy = dy * act.abs() + y.abs() * (act.abs() * (rel_act + 2 * E32) + far)
        y = y * act
    return y, 1.01 * (dy + y.abs() * half_step(kind)) + tiny_step(kind)


def exactly(got, want, what):
    """Equal numbers, NaN where NaN is wanted."""
    got, want = got.double().cpu(), want.double()
    bad = ~((got == want) | (torch.isnan(got) & torch.isnan(want)))
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} differ, first at {bad.nonzero()[0].tolist()}"

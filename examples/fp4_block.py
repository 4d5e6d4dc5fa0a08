"""A softmax block over a cache in 4 bits, from residual stream to residual stream, as a model calls it.

`Fp4Block.forward` takes the stream's normed rows, projects them, norms and rotates queries and keys, writes the new keys and
values into the cache, attends over it, gates the heads, and hands its output to the norm that adds it to the stream: for
whole prompts and for single tokens alike.  A decode step is captured into a graph and replayed.

    python examples/fp4_block.py        # needs the GPU; prints what it checked
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_delta_rule_varlen_amd as gdn  # noqa: E402


class Fp4Block:
    """Projections, norms and a 4-bit cache of `room` rows a sequence."""

    def __init__(self, width, H, HK, D, batch, room, *, dtype=torch.bfloat16, device="cuda", seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)
        normal = lambda *shape: torch.randn(shape, generator=gen, device=device, dtype=torch.float32)
        self.H, self.HK, self.D, self.dtype, self.device = H, HK, D, dtype, device
        self.parts = [H * D, HK * D, HK * D, H * D]  # queries, keys, values, gate
        self.w_in = (normal(width, sum(self.parts)) / width**0.5).to(dtype)
        self.w_out = (normal(H * D, width) / (H * D) ** 0.5).to(dtype)
        self.q_weight, self.k_weight, self.head_weight = (1 + 0.1 * normal(D) for _ in range(3))
        self.post_weight, self.next_weight = 1 + 0.1 * normal(width), 1 + 0.1 * normal(width)
        self.inv_freq = 1e4 ** (-torch.arange(0, D, 2, device=device, dtype=torch.float32) / D)
        self.cache = gdn.fp4_cache(batch * room, HK, D, device=device)
        self.begin = torch.arange(batch, device=device) * room
        self.past = torch.zeros(batch, dtype=torch.int32, device=device)

    def forward(self, x, residual, offsets, new, max_q, attend=None):
        """x [N, width]: normed rows of the stream `residual` [N, width] (fp32); `new` int32 [batch]: tokens of every sequence.
        Returns the normed rows of the stream behind the block, and the stream."""
        q, k, v, gate = (p.unflatten(1, (-1, self.D)) for p in (x @ self.w_in).split(self.parts, dim=1))
        q, k, _ = gdn.qk_norm_rope_varlen(q, k, None, offsets, inv_freq=self.inv_freq, q_weight=self.q_weight,
                                          k_weight=self.k_weight, positions=self.past)
        gdn.cache_write_fp4_varlen(k, v, offsets, cache=self.cache, past=self.past, kv_begin=self.begin)
        self.past += new
        o = (attend or self.attend)(q, offsets, max_q)
        o = gdn.gated_norm(o, gate, weight=self.head_weight, activation="sigmoid", out=o)
        return gdn.residual_norm(o.flatten(1) @ self.w_out, residual, weight=self.next_weight, post_weight=self.post_weight,
                                 scale=0.5, residual_out=residual)

    def attend(self, q, offsets, max_q):
        return gdn.attention_fp4_varlen(q, self.cache, offsets, kv_len=self.past, kv_begin=self.begin, max_q=max_q)[0]

    def attend_plainly(self, q, offsets, max_q):
        """The same over a plain copy of what the cache stands for."""
        rows = self.cache.k_codes.shape[0]
        whole = torch.tensor([0, rows], dtype=torch.int32, device=self.device)
        k, v = gdn.cache_read_fp4_varlen(self.cache, whole, N=rows, dtype=self.dtype)
        return gdn.attention_varlen(q, k, v, offsets, kv_len=self.past, kv_begin=self.begin, max_q=max_q)[0]


def main():
    torch.manual_seed(0)
    width, prompts, steps = 256, [37, 5, 260, 0, 64], 3
    batch = len(prompts)
    make = lambda: Fp4Block(width, H=8, HK=2, D=64, batch=batch, room=512)
    ints = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    streams = [torch.randn(t + steps, width, device="cuda") for t in prompts]

    def enter(rows):  # the norm before the block
        return gdn.residual_norm(rows.to(torch.bfloat16), write_residual=False)[0]

    def prompt(block, lengths, attend=None):
        residual = torch.cat([s[:t] for s, t in zip(streams, lengths)])
        offsets = torch.nn.functional.pad(ints(lengths).cumsum(0, dtype=torch.int32), (1, 0))
        return block.forward(enter(residual), residual.clone(), offsets, ints(lengths), max(lengths), attend)

    # prompts, over the 4-bit cache and over a plain copy of it
    block, plain = make(), make()
    got = [prompt(block, prompts)]
    want = prompt(plain, prompts, plain.attend_plainly)
    for a, b in zip(got[0], want):
        torch.testing.assert_close(a.float(), b.float(), rtol=5e-2, atol=5e-2)

    # single tokens: one step captured, and replayed with the next tokens in the same buffers
    residual = torch.empty(batch, width, device="cuda")
    x = torch.empty(batch, width, device="cuda", dtype=torch.bfloat16)
    offsets, one = torch.arange(batch + 1, dtype=torch.int32, device="cuda"), ints([1] * batch)
    graph, past = torch.cuda.CUDAGraph(), block.past.clone()
    with torch.cuda.graph(graph):
        out = block.forward(x, residual, offsets, one, 1)
    block.past.copy_(past)  # a capture runs nothing
    for i in range(steps):
        residual.copy_(torch.stack([s[t + i] for s, t in zip(streams, prompts)]))
        x.copy_(enter(residual))
        graph.replay()
        got.append([y.clone() for y in out])
    torch.cuda.synchronize()

    # the same tokens in one call on a fresh cache
    lengths = [len(s) for s in streams]
    once = [y.split(lengths) for y in prompt(make(), lengths)]
    for b, t in enumerate(prompts):
        at = sum(prompts[:b])
        for j in range(2):
            parts = torch.cat([got[0][j][at:at + t]] + [g[j][b:b + 1] for g in got[1:]])
            torch.testing.assert_close(parts.float(), once[j][b].float(), rtol=5e-2, atol=5e-2)
    print("prompts, replayed single tokens and a plain copy of the cache agree", flush=True)


if __name__ == "__main__":
    main()

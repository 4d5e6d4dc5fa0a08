"""The softmax-attention operators as a model calls them, one layer of them over a cache.

A batch of packed prompts is answered token by token: `attend` norms and rotates the new queries and keys, writes
keys and values into the cache and attends over it, for whole prompts and for single tokens alike.  Then
several continuations of the first conversation share its cache rows as a prefix that is read once for all.

    python examples/softmax_layer.py        # needs the GPU; prints what it checked
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_delta_rule_varlen_amd as gdn  # noqa: E402


class SoftmaxLayer:
    """Projections, per-head norms, rotary positions and a cache of `room` rows a sequence."""

    def __init__(self, width, H, HK, D, rot, batch, room, *, dtype=torch.bfloat16, device="cuda", seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)
        normal = lambda *shape: torch.randn(shape, generator=gen, device=device, dtype=torch.float32)
        self.H, self.HK, self.D, self.dtype, self.device = H, HK, D, dtype, device
        self.w_in = (normal(width, (H + 2 * HK) * D) / width**0.5).to(dtype)
        self.w_out = (normal(H * D, width) / (H * D) ** 0.5).to(dtype)
        self.q_weight, self.k_weight = 1 + 0.1 * normal(D), 1 + 0.1 * normal(D)
        self.inv_freq = 1e4 ** (-torch.arange(0, rot, 2, device=device, dtype=torch.float32) / rot)
        self.k, self.v = (torch.zeros((batch * room, HK, D), dtype=dtype, device=device) for _ in range(2))
        self.begin = torch.arange(batch, device=device) * room
        self.past = torch.zeros(batch, dtype=torch.int32, device=device)

    def project(self, x):
        """(q, k, v) of the tokens x [N, width], as views of one packed row each."""
        row = x.to(self.dtype) @ self.w_in
        q, k, v = row.split([self.H * self.D, self.HK * self.D, self.HK * self.D], dim=1)
        return q.unflatten(1, (self.H, self.D)), k.unflatten(1, (self.HK, self.D)), v.unflatten(1, (self.HK, self.D))

    def attend(self, x, lengths):
        """The layer over `lengths[b]` new tokens of every sequence b (x packed, [N, width]); the cache grows by them."""
        T = torch.tensor(lengths, dtype=torch.int32, device=self.device)
        offsets = torch.nn.functional.pad(T.cumsum(0, dtype=torch.int32), (1, 0))
        q, k, v = self.project(x)
        q, _, _ = gdn.qk_norm_rope_varlen(q, k, v, offsets, inv_freq=self.inv_freq, q_weight=self.q_weight,
                                          k_weight=self.k_weight, past=self.past, kv_begin=self.begin, k_out=self.k,
                                          v_out=self.v)
        self.past += T
        out, _ = gdn.attention_varlen(q, self.k, self.v, offsets, kv_len=self.past, kv_begin=self.begin, max_q=max(lengths))
        return out.flatten(1) @ self.w_out

    def continue_shared(self, x, prefix_len):
        """One new token for each of len(x) continuations of the first `prefix_len` rows of sequence 0; each one's own
        keys are its token's alone."""
        n = len(x)
        offsets = torch.arange(n + 1, dtype=torch.int32, device=self.device)
        q, k, v = self.project(x)
        at = torch.full((n,), prefix_len, dtype=torch.int32, device=self.device)
        # without kv_begin the rows are the tokens' own, and `positions` alone places them
        q, k, v = gdn.qk_norm_rope_varlen(q, k, v, offsets, inv_freq=self.inv_freq, q_weight=self.q_weight,
                                          k_weight=self.k_weight, positions=at)
        out, _ = gdn.attention_prefix_varlen(q, self.k[:prefix_len], self.v[:prefix_len], k, v, offsets, max_q=1)
        return out.flatten(1) @ self.w_out


def main():
    torch.manual_seed(0)
    width, prompts = 256, [37, 5, 260, 0, 64]
    layer = SoftmaxLayer(width, H=8, HK=2, D=64, rot=32, batch=len(prompts), room=512)
    x = [torch.randn(t + 3, width, device="cuda", dtype=torch.bfloat16) for t in prompts]

    # prompts at once, then three tokens each
    steps = [layer.attend(torch.cat([s[:t] for s, t in zip(x, prompts)]), prompts)]
    for i in range(3):
        steps.append(layer.attend(torch.stack([s[t + i] for s, t in zip(x, prompts)]), [1] * len(prompts)))

    # the same tokens in one call on a fresh cache
    whole = SoftmaxLayer(width, H=8, HK=2, D=64, rot=32, batch=len(prompts), room=512)
    once = whole.attend(torch.cat(x), [len(s) for s in x]).split([len(s) for s in x])
    for b, t in enumerate(prompts):
        begin = sum(prompts[:b])
        parts = torch.cat([steps[0][begin:begin + t]] + [s[b:b + 1] for s in steps[1:]])
        torch.testing.assert_close(parts, once[b], rtol=2e-2, atol=2e-2)

    # four continuations of sequence 0, which share its rows
    tokens = torch.randn(4, width, device="cuda", dtype=torch.bfloat16)
    shared = layer.continue_shared(tokens, prefix_len=40)
    single = SoftmaxLayer(width, H=8, HK=2, D=64, rot=32, batch=4, room=64)
    for b in range(4):
        single.k[64 * b:64 * b + 40], single.v[64 * b:64 * b + 40] = layer.k[:40], layer.v[:40]
    single.past += 40
    torch.testing.assert_close(shared, single.attend(tokens, [1] * 4), rtol=2e-2, atol=2e-2)
    print("prompts, single tokens and shared prefixes agree", flush=True)


if __name__ == "__main__":
    main()

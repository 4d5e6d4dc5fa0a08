"""A block over a cache in 4 bits, its operators together as a model calls them: the example runs, and a block's stages are each
what their formulas give on the stage before."""
import importlib.util
import os

import pytest

from attn_util import assert_within, attention_ref, rope_ref
from fp4_util import decode, encode, exactly, gated_ref, residual_ref
from gpu_util import ensure_built, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    ensure_built()
    return require_gpu()


def example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "fp4_block.py")
    spec = importlib.util.spec_from_file_location("fp4_block", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_example_runs(torch):
    example().main()


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
def test_stages(torch, kind):
    """The block's calls in their order, each against its formula on what the call before it left."""
    import gated_delta_rule_varlen_amd as gdn
    from attn_util import DT

    gen = torch.Generator().manual_seed(7)
    normal = lambda *s: torch.randn(s, generator=gen).to(DT[kind])
    H, HK, D, T, past, room = 6, 2, 64, [3, 1, 0, 9], [5, 40, 7, 0], 60
    N, off = sum(T), [0, 3, 4, 4, 13]
    ints = lambda x, t=torch.int32: torch.tensor(x, dtype=t, device="cuda")
    offsets, begin = ints(off), [room * b for b in range(4)]
    q, k, v, gate = (normal(N, h, D) for h in (H, HK, HK, H))
    weight, freq = 1 + 0.1 * torch.randn(D, generator=gen), 1e4 ** (-torch.arange(0, D, 2).float() / D)
    cache = gdn.fp4_cache(4 * room, HK, D)
    old = [normal(sum(past), HK, D) for _ in range(2)]
    at = dict(cache=cache, kv_begin=ints(begin, torch.int64))
    gdn.cache_write_fp4_varlen(*(x.cuda() for x in old), ints([0, 5, 45, 52, 52]), **at)

    q1, k1, _ = gdn.qk_norm_rope_varlen(q.cuda(), k.cuda(), None, offsets, inv_freq=freq.cuda(), q_weight=weight.cuda(),
                                        k_weight=weight.cuda(), positions=ints(past))
    pos = torch.cat([torch.arange(t) + p for t, p in zip(T, past)])
    for got, x in ((q1, q), (k1, k)):
        ref = rope_ref(x, weight, pos, freq, eps=1e-6, interleaved=False, kind=kind)
        assert_within(got, ref[0], ref[1], f"{kind} rotated")

    gdn.cache_write_fp4_varlen(k1, v.cuda(), offsets, past=ints(past), **at)
    n = [t + p for t, p in zip(T, past)]
    rk, rv = gdn.cache_read_fp4_varlen(cache, offsets, N=N, past=ints(past), kv_begin=at["kv_begin"], dtype=DT[kind])
    exactly(rk, decode(*encode(k1.cpu(), kind)), f"{kind} keys")
    exactly(rv, decode(*encode(v, kind)), f"{kind} values")

    o, _ = gdn.attention_fp4_varlen(q1, cache, offsets, kv_len=ints(n), kv_begin=at["kv_begin"], max_q=9)
    held = [decode(*(x.cpu() for x in cache[2 * i:2 * i + 2])) for i in range(2)]
    ref = attention_ref(q1.cpu(), *held, T, begin, n, kind=kind)
    lost = 2.0 ** -126 * max(n) * held[1].abs().max()  # exponentials below fp32's normal range are zeros
    assert_within(o, ref[0], (3.0 if kind == "f32" else 1.0) * ref[2] + lost, f"{kind} attention")

    g = gdn.gated_norm(o, gate.cuda(), weight=weight.cuda())
    ref = gated_ref(o.cpu(), gate, weight, 1e-6, "silu", False, True, kind)
    assert_within(g, ref[0], ref[1], f"{kind} gated")

    stream, w = torch.randn(N, H * D, generator=gen), 1 + 0.1 * torch.randn(H * D, generator=gen)
    out, nxt = gdn.residual_norm(g.flatten(1), stream.cuda(), weight=w.cuda(), post_weight=w.cuda(), scale=0.5)
    ref = residual_ref(g.cpu().flatten(1), stream, w, w, 0.5, None, 1e-6, kind, "f32")
    assert_within(out, ref[0], ref[2], f"{kind} out")
    assert_within(nxt, ref[1], ref[3], f"{kind} stream")

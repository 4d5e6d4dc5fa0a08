"""GPU tests of the 4-bit cache: what is written equals the reference byte for byte, and reads back as its values."""
import pytest

from attn_util import DT, layout
from fp4_util import decode, encode, exactly, strided
from gpu_util import ensure_built, require_gpu

pytestmark = pytest.mark.gpu
I32 = dict(device="cuda")


@pytest.fixture(scope="module")
def torch():
    ensure_built()
    return require_gpu()


def offsets_of(torch, T):
    off = [0]
    for t in T:
        off.append(off[-1] + t)
    return torch.tensor(off, dtype=torch.int32, device="cuda")


def filled(torch, rows, HK, D, kind, byte=0xA5):
    """A cache whose bytes are all `byte`, in one of three layouts."""
    parts = [torch.full((rows, HK, w), byte, dtype=torch.uint8) for w in (D // 2, D // 32, D // 2, D // 32)]
    return tuple(strided(p, kind) for p in parts)


def check(torch, kind, HK, D, lengths, cache_layout="heads", token_layouts=("rows", "rows"), runs=True, k=None, v=None, seed=3):
    """lengths: (new tokens, tokens already there) per sequence."""
    import gated_delta_rule_varlen_amd as gdn

    gen = torch.Generator().manual_seed(seed)
    T, past = [t for t, _ in lengths], [p for _, p in lengths]
    N = sum(T)
    if k is None:
        k, v = ((torch.randn(N, HK, D, generator=gen) * torch.exp2(torch.randint(-6, 6, (N, HK, 1), generator=gen))).to(DT[kind])
                for _ in range(2))
    if runs:
        begin, rows = layout([(t, t + p) for t, p in lengths])
        place = torch.cat([torch.arange(t) + b + p for b, t, p in zip(begin, T, past)]) if N else torch.zeros(0, dtype=torch.long)
    else:
        begin, rows, place = None, N + 5, torch.arange(N)
    cache = filled(torch, rows, HK, D, cache_layout)
    want = [x.cpu().clone() for x in cache]
    (want[0][place], want[1][place]), (want[2][place], want[3][place]) = encode(k, kind), encode(v, kind)
    at = {} if not runs else dict(kv_begin=torch.tensor(begin, dtype=torch.int64, device="cuda"),
                                  past=torch.tensor(past, dtype=torch.int32, device="cuda"))
    off, status = offsets_of(torch, T), torch.full((1,), 9, dtype=torch.int32, device="cuda")
    got = gdn.cache_write_fp4_varlen(strided(k, token_layouts[0]), strided(v, token_layouts[1]), off, cache=cache, dev_status=status, **at)
    assert got is cache and status.item() == 0
    for x, y, name in zip(cache, want, ("k codes", "k scales", "v codes", "v scales")):
        assert torch.equal(x.cpu(), y), f"{kind} HK={HK} D={D} {name}: {(x.cpu() != y).nonzero()[:3].tolist()}"
    for dtype in (DT[kind], torch.float32):
        rk, rv = gdn.cache_read_fp4_varlen(cache, off, N=N, dtype=dtype, dev_status=status, **at)
        exactly(rk, decode(*encode(k, kind)), f"{kind} keys back as {dtype}")
        exactly(rv, decode(*encode(v, kind)), f"{kind} values back as {dtype}")
    out = torch.full((N, HK, 3 * D), 7.0, dtype=DT[kind], device="cuda")  # into parts of wider rows
    rk, rv = gdn.cache_read_fp4_varlen(cache, off, k_out=out[:, :, :D], v_out=out[:, :, 2 * D:], **at)
    exactly(rk, decode(*encode(k, kind)), "strided keys back")
    exactly(rv, decode(*encode(v, kind)), "strided values back")
    assert (out[:, :, D:2 * D] == 7.0).all()


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D", [32, 64, 96, 128, 160, 192, 224, 256])
def test_widths(torch, kind, D):
    check(torch, kind, 3, D, [(5, 2), (0, 4), (1, 0), (40, 7)])


@pytest.mark.parametrize("cache_layout", ["rows", "heads", "wide"])
@pytest.mark.parametrize("token_layouts", [("rows", "heads"), ("wide", "wide"), ("heads", "rows")])
def test_layouts(torch, cache_layout, token_layouts):
    check(torch, "bf16", 4, 64, [(3, 1), (17, 0)], cache_layout, token_layouts)
    check(torch, "f32", 1, 96, [(3, 1), (17, 0)], cache_layout, token_layouts, runs=False)


@pytest.mark.parametrize("lengths", [[(1, 0)], [(0, 3)], [(0, 0), (0, 0)], [(1, 5)] * 300, [(4000, 0), (1, 9), (700, 50)],
                                     [(0, 1), (9, 0), (0, 0)]])
def test_lengths(torch, lengths):
    check(torch, "bf16", 2, 128, lengths)
    check(torch, "f16", 1, 32, lengths)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_every_number(torch, kind):
    """All bit patterns of the type (infinities and NaN among them), in the order they count and shuffled."""
    x = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(DT[kind]).view(-1, 1, 64)
    y = x.flatten()[torch.randperm(1 << 16, generator=torch.Generator().manual_seed(1))].view(-1, 1, 64)
    check(torch, kind, 1, 64, [(1024, 0)], k=x, v=y)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
def test_borders(torch, kind):
    """Ties between codes and their neighbours in the type, in blocks of every power and both signs."""
    eps = torch.finfo(DT[kind]).eps
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    block = torch.cat((mid, mid * (1 - eps / 2), mid * (1 + eps), torch.tensor([6.0, 0.0, 0.5, 5.9])))
    block = torch.cat((block, -block[:7]))
    lo, hi = {"bf16": (-120, 120), "f32": (-120, 120), "f16": (-10, 13)}[kind]
    x = torch.stack([block * 2.0**e for e in range(lo, hi)]).to(DT[kind])
    x = torch.cat((x, x.flip(1)), dim=1).view(-1, 1, 64)
    top = torch.tensor([6.0, 6 * (1 + eps), 3.0, 3 * (1 + eps)])  # the largest element around a change of power
    y = torch.zeros(len(x), 1, 64)
    y[:, 0, 0], y[:, 0, 40], y[:, 0, 9] = 1.0, -top.repeat(len(x))[: len(x)], top.repeat(len(x))[: len(x)]
    check(torch, kind, 1, 64, [(len(x), 0)], k=x, v=y.to(DT[kind]))


def test_large_fp16_numbers_become_the_largest_value(torch):
    x = torch.tensor([65504.0, -49152.0, 50000.0, -65504.0] * 16).half().view(1, 1, 64)
    check(torch, "f16", 1, 64, [(1, 0)], k=x, v=x / 3)


def test_rows_past_32_bits(torch):
    """A run whose bytes begin past 2^32."""
    import gated_delta_rule_varlen_amd as gdn

    HK, D, rows = 2, 256, (1 << 32) // 256 + 100
    cache = gdn.fp4_cache(rows, HK, D)
    assert cache.k_codes.transpose(0, 1).is_contiguous()
    gen = torch.Generator().manual_seed(1)
    k, v = (torch.randn(3, HK, D, generator=gen).bfloat16() for _ in range(2))
    off, begin = offsets_of(torch, [3]), torch.tensor([rows - 5], dtype=torch.int64, device="cuda")
    gdn.cache_write_fp4_varlen(k.cuda(), v.cuda(), off, cache=cache, kv_begin=begin)
    rk, rv = gdn.cache_read_fp4_varlen(cache, off, N=3, kv_begin=begin)
    exactly(rk, decode(*encode(k, "bf16")), "keys")
    exactly(rv, decode(*encode(v, "bf16")), "values")
    assert (cache.k_codes[: rows - 5] != 0).sum() == 0 and (cache.v_scales[rows - 2:] != 0).sum() == 0


def test_the_binding_refuses_a_bad_cache(torch):
    import gated_delta_rule_varlen_amd as gdn

    c, off = gdn.fp4_cache(9, 2, 64), offsets_of(torch, [4])
    x = torch.zeros(4, 2, 64, device="cuda")
    at = dict(kv_len=off[1:], kv_begin=torch.zeros(1, dtype=torch.int64, device="cuda"))
    bad = [c[:3], iter(c), tuple(t.cpu() for t in c), c._replace(v_scales=c.v_scales[:5]), c._replace(k_codes=c.k_codes.int()),
           c._replace(k_scales=c.k_scales[:, :1]), c._replace(v_codes=c.v_codes[:, :, :16]), [None] * 4,
           c._replace(k_codes=torch.zeros(9, 2, 64, dtype=torch.uint8, device="cuda")[:, :, ::2])]
    for cache in bad:
        for call in (lambda: gdn.cache_write_fp4_varlen(x, x, off, cache=cache), lambda: gdn.cache_read_fp4_varlen(cache, off, N=4),
                     lambda: gdn.cache_read_fp4_varlen(cache, off, k_out=x), lambda: gdn.attention_fp4_varlen(x, cache, off, **at)):
            with pytest.raises((TypeError, ValueError)):
                call()
    with pytest.raises((TypeError, ValueError)):
        gdn.cache_read_fp4_varlen(c, off, N=4, dtype=torch.float64)
    with pytest.raises(gdn.GdnError):
        gdn.attention_fp4_varlen(x, c, off, kv_len=None, kv_begin=None)
    with pytest.raises(ValueError):  # three heads of a cache with two
        gdn.cache_write_fp4_varlen(torch.zeros(4, 3, 64, device="cuda"), torch.zeros(4, 3, 64, device="cuda"), off, cache=c)


@pytest.mark.parametrize("bad", ["first", "last", "falls", "past", "begin", "end"])
def test_malformed_calls_write_nothing(torch, bad):
    import gated_delta_rule_varlen_amd as gdn

    off = {"first": [1, 3, 8], "last": [0, 3, 7], "falls": [0, 9, 8]}.get(bad, [0, 3, 8])
    past, begin = [0, 2], [0, 10]
    if bad == "past":
        past[1] = -1
    if bad == "begin":
        begin[0] = -1
    if bad == "end":
        begin[1] = 14  # rows 16 .. 20 of 20
    dev = lambda x, t: torch.tensor(x, dtype=t, device="cuda")
    at = dict(past=dev(past, torch.int32), kv_begin=dev(begin, torch.int64))
    cache = filled(torch, 20, 2, 64, "rows")
    x, status = torch.randn(8, 2, 64, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.cache_write_fp4_varlen(x, x, dev(off, torch.int32), cache=cache, dev_status=status, **at)
    assert status.item() == -9 and all((c == 0xA5).all() for c in cache)
    out = torch.full((2, 8, 2, 64), 7.0, device="cuda")
    status.zero_()
    gdn.cache_read_fp4_varlen(cache, dev(off, torch.int32), k_out=out[0], v_out=out[1], dev_status=status, **at)
    assert status.item() == -9 and (out == 7.0).all()


def test_write_and_read_in_a_graph(torch):
    import gated_delta_rule_varlen_amd as gdn

    gen = torch.Generator().manual_seed(5)
    x = [torch.randn(6, 2, 128, generator=gen).bfloat16().cuda() for _ in range(3)]
    k, v = x[0].clone(), x[1].clone()
    cache = gdn.fp4_cache(6, 2, 128)
    off = offsets_of(torch, [6])
    out = torch.empty(2, 6, 2, 128, dtype=torch.bfloat16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.cache_write_fp4_varlen(k, v, off, cache=cache)
        gdn.cache_read_fp4_varlen(cache, off, k_out=out[0], v_out=out[1])
    for i in range(3):
        k.copy_(x[i])
        v.copy_(x[(i + 1) % 3])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        exactly(out[0], decode(*encode(x[i].cpu(), "bf16")), "keys")
        exactly(out[1], decode(*encode(x[(i + 1) % 3].cpu(), "bf16")), "values")

"""GPU tests of attention_fp4_varlen where a cache's scales leave the range of the operands.  With fp16 queries values are
operands in fp16, so those of scale bytes from 141 on may be infinite (6 * 2^14 is); with the others, whose operands have
fp32's range, those of 253 and 254."""
import pytest

from attn_util import DT, E32, assert_within, attention_ref
from fp4_util import decode, exactly, strided
from gpu_util import ensure_built, require_gpu
from test_gpu_fp4_attention import Case

pytestmark = pytest.mark.gpu

# head width, query heads of a key head, (new tokens, cache rows) per sequence: a block a run; runs cut and joined; row tiles
# that share a block; two groups of waves; heads divided among blocks; prompts of every width
FORMS = [(64, 4, [(4, 40), (4, 300)]), (128, 4, [(4, 3000), (3, 77)]), (128, 8, [(5, 3000), (2, 40)]), (256, 8, [(5, 4000), (2, 40)]),
         (192, 8, [(9, 400), (2, 30)]), (64, 4, [(70, 170)]), (128, 4, [(90, 300)]), (256, 4, [(90, 300), (40, 70)])]
# Small scores: the smallest probability is a normal number of every type.  |q k| <= 6 |q| summed over a head stays below 8
# in exponents of two.
SCALE = 2.0 ** -10


@pytest.fixture(scope="module")
def torch():
    ensure_built()
    return require_gpu()


def operands(torch, c):
    """The cache's values as the kernels multiply them: fp16 with fp16 queries, otherwise exact or past fp32's range."""
    t = torch.float16 if c.kind == "f16" else torch.float32
    return [x.to(t).double() for x in c.values()]


def check(torch, c, what):
    """Against the 64-bit form over the operands; what is infinite or no number there is so here, and nothing else."""
    import gated_delta_rule_varlen_amd as gdn

    k, v = operands(torch, c)
    ref, _, tol, _ = attention_ref(c.q, k, v, c.T, c.begin, c.n, kind=c.kind, scale=SCALE)
    by = 3.0 if c.kind == "f32" else 1.0  # three parts, as in the tests beside these
    for max_q in (max(c.T), 1000):  # the call's own form, and that of prompts
        out = gdn.attention_fp4_varlen(**c.dev(), max_q=max_q, scale=SCALE)[0].double().cpu()
        sound = torch.isfinite(ref)
        assert (torch.isfinite(out) == sound).all(), f"{what} max_q {max_q}: {int((torch.isfinite(out) != sound).sum())} differ"
        assert (torch.isnan(out) == torch.isnan(ref)).all() and (out[torch.isinf(ref)] == ref[torch.isinf(ref)]).all()
        assert_within(out[sound], ref[sound], by * tol[sound], f"{what} max_q {max_q}")


@pytest.mark.parametrize("which", ["keys", "values"])
@pytest.mark.parametrize("D,G,lengths", FORMS)
def test_infinite_operands_in_rows_done_again(torch, which, D, G, lengths):
    """An infinity of fp16 in the first row of each sequence, which all tokens see, and a value without a number in the last
    row, for which the rows before it are done again."""
    c = Case(torch, "f16", 2, G, D, lengths)
    scales = 1 if which == "keys" else 3
    for b, n in enumerate(c.n):
        c.cache[scales][c.begin[b], 0, 1] = 141
        c.cache[scales - 1][c.begin[b], 0, 16:32] = 0x77
        c.cache[3][c.begin[b] + n - 1, 0, 0] = 255
    check(torch, c, f"{which} {D}")


@pytest.mark.parametrize("kind,byte", [("f16", 141), ("f16", 150), ("f16", 252), ("f16", 254), ("bf16", 253), ("bf16", 254), ("f32", 253),
                                       ("f32", 254)])
@pytest.mark.parametrize("D,G,lengths", FORMS)
def test_infinite_values_behind_a_mask(torch, kind, byte, D, G, lengths):
    """In the last row of each sequence, which only the last token sees."""
    c = Case(torch, kind, 2, G, D, lengths)
    for b, n in enumerate(c.n):
        c.cache[3][c.begin[b] + n - 1, 0, 1] = byte
        c.cache[2][c.begin[b] + n - 1, 0, 16:32] = 0x77
    check(torch, c, f"{kind} {byte} {D}")


def every_byte(torch, low, high, rows, places, gen):
    """Scale bytes [rows, places]: each place has every byte of low .. high, beside bytes drawn for the others."""
    some = torch.arange(rows) % (high - low + 1) + low
    return torch.stack([some[torch.randperm(rows, generator=gen)] for _ in range(places)], dim=1).byte()


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D", [32, 64, 96, 128, 256])
@pytest.mark.parametrize("layout", ["rows", "heads", "wide", "odd"])
@pytest.mark.parametrize("room", [0, 60000])
def test_every_scale_beside_any_other(torch, kind, D, layout, room):
    """A kernel may read four scales at a time and hand an instruction one of them with its neighbours' bits beside it.  One key a
    sequence with a query of zeros: the output is the value itself, exactly, as it is a number of every type.  Then a query
    that picks one element of each block and undoes its power: the log of the sum is the code's value, to the roundings of
    the scale to base 2, the product, the logarithm and the way back (two units each; in fp16 the maximum is kept lower by
    four, and they are of that much more).  Powers are those of which all values are normal numbers of the type, and of
    which the undoing ones are.  "odd": scales that lie at odd addresses."""
    import gated_delta_rule_varlen_amd as gdn

    low, high, lower = (114, 140, 4.0) if kind == "f16" else (2, 252, 0.0)
    gen = torch.Generator().manual_seed(D)
    NB, some, rows = D // 32, 251, 1004
    codes = [torch.randint(0, 256, (rows, 1, D // 2), generator=gen, dtype=torch.uint8) for _ in range(2)]
    scales = [every_byte(torch, low, high, rows, NB, gen).view(rows, 1, NB) for _ in range(2)]
    cache = []
    for part in (codes[0], scales[0], codes[1], scales[1]):  # rows of no sequence behind: then runs are cut and joined
        part = torch.cat([part, torch.full((room, 1, part.shape[2]), 255, dtype=torch.uint8)])
        if layout == "odd" and part.shape[2] == NB:
            cache.append(torch.nn.functional.pad(part, (1, NB % 2)).cuda()[:, :, 1:1 + NB])
        else:
            cache.append(strided(part, "rows" if layout == "odd" else layout))
    ints = lambda x, t=torch.int32: x.to(t).cuda()
    offsets, kv_len = ints(torch.arange(some + 1)), ints(torch.ones(some))
    q = torch.zeros(rows, NB, D, dtype=torch.float64)  # head h: one element of block h, at another place in each row
    h, i = torch.arange(NB), torch.arange(rows)[:, None]
    place = 32 * h + (i + 5 * h) % 32
    q[i, h, place] = 2.0 ** (127 - scales[0][:, 0].double())
    v, want = decode(codes[1], scales[1]), decode(codes[0], scales[0])[:, 0].gather(1, place) * q[i, h, place]
    q = q.to(DT[kind]).cuda()
    for first in range(0, rows, some):
        part = slice(first, first + some)
        at = dict(kv_len=kv_len, kv_begin=ints(torch.arange(first, first + some), torch.int64))
        for max_q in (1, 300):
            out, _ = gdn.attention_fp4_varlen(torch.zeros_like(q[part]), cache, offsets, max_q=max_q, **at)
            exactly(out, v[part].expand(some, NB, D), f"values {kind} {D}")
            _, lse = gdn.attention_fp4_varlen(q[part], cache, offsets, max_q=max_q, scale=1.0, return_lse=True, **at)
            assert_within(lse, want[part], 8 * E32 * (want[part].abs() + lower), f"keys {kind} {D}")


# head width, key heads, query heads of each, tokens, rows of the cache without a sequence, max_q: a block a run, cut runs, several row
# tiles, prompts
EXACT = [(64, 2, 4, 1, 0, 1), (64, 2, 4, 1, 90000, 1), (128, 2, 16, 3, 90000, 3), (256, 1, 8, 2, 90000, 2), (64, 2, 2, 1, 0, 400),
                 (128, 1, 4, 1, 0, 400), (256, 1, 2, 1, 0, 400)]


@pytest.mark.parametrize("D,HK,G,T,room,max_q", EXACT)
def test_single_precision_keeps_all_its_bits(torch, D, HK, G, T, room, max_q):
    """fp32 queries and probabilities are multiplied in parts; here a part that is lost shows, as nothing else is rounded much.
    Two keys a sequence: zeros with values of ones, and one element of 1 with a value of zeros; queries of one element
    x in (0, 1) with all 24 bits.  The second score is scale * x, exactly as the parts are a sum; out = 1 / (1 + exp(scale x)).
    Its argument to base 2 is off by the scale's, the product's and the maximum's roundings (3 e |s| each way), the
    exponential by 2 e, the sum, its reciprocal (2 e) and the product by 4 e, a part's own rest by 2^-27: 8 e |s| + 10 e in
    all.  lse is off by the scale, the product, the constant and the sum (8 e of itself and 8 e)."""
    import gated_delta_rule_varlen_amd as gdn

    B, gen = 40, torch.Generator().manual_seed(D + T)
    codes = [torch.zeros(2 * B + room, HK, D // 2, dtype=torch.uint8) for _ in range(2)]
    scales = torch.full((2 * B + room, HK, D // 32), 127, dtype=torch.uint8)
    scales[2 * B:] = 255
    at = 5
    codes[0][1:2 * B:2, :, at // 2] = 0x20  # the element's code, 1
    codes[1][0:2 * B:2] = 0x22              # the first key's values, ones
    cache = [strided(x, "heads") for x in (codes[0], scales, codes[1], scales)]
    x = torch.rand(B * T, HK * G, generator=gen)
    q = torch.zeros(B * T, HK * G, D)
    q[:, :, at] = x
    ints = lambda x, t=torch.int32: x.to(t).cuda()
    out, lse = gdn.attention_fp4_varlen(q.cuda(), cache, ints(torch.arange(B + 1) * T), kv_len=ints(torch.full((B,), 2)),
                                        kv_begin=ints(2 * torch.arange(B), torch.int64), max_q=max_q, scale=1.0, return_lse=True)
    last = torch.arange(T - 1, B * T, T)  # a sequence's last token sees both

    def forms(y, drop=lambda p: p):
        p = drop(torch.exp(-y))  # against the larger score
        return p / (1 + torch.exp(-y)), y + torch.log1p(torch.exp(-y))

    def two_parts(y):
        first = y.float().bfloat16().double()
        return first + (y - first).float().bfloat16().double()

    s = x[last].double()
    ref, ref_lse = forms(s)
    tol, tol_lse = (8 * s + 10) * E32 * ref, 8 * E32 * (ref_lse + 1)
    assert_within(out.cpu()[last], ref[..., None].expand(-1, -1, D), tol[..., None], f"out {D}")
    assert_within(lse.cpu()[last], ref_lse, tol_lse, f"lse {D}")
    # without the third part of the probabilities or the queries these bounds are passed
    assert ((forms(s, two_parts)[0] - ref).abs() > 1.5 * tol).any()
    assert ((forms(two_parts(s))[1] - ref_lse).abs() > 1.0 * tol_lse).any()

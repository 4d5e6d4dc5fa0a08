"""GPU tests of attention_fp4_varlen against a plain 64-bit attention over the values the cache stands for: types, head widths
and layouts, lengths around every tile edge, rows without keys, blocks without numbers in places that are masked, long
runs cut in parts, malformed calls, streams and graphs."""
import math
import random

import pytest

from attn_util import DT, assert_within, attention_ref, layout
from fp4_util import decode, strided
from gpu_util import bits, ensure_built, require_gpu, sentinel

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    ensure_built()
    return require_gpu()


class Case:
    """Seeded inputs: lengths are (new tokens, cache rows) per sequence.  The cache's bytes are drawn: any codes, and powers of
    which a head's differ by up to 2^4; rows of no sequence read as NaN."""

    def __init__(self, torch, kind, HK, G, D, lengths, cache_layout="heads", seed=1, q_layout="rows", powers=(124, 127)):
        self.torch, self.kind, self.lengths = torch, kind, lengths
        gen = torch.Generator().manual_seed(seed)
        order = list(range(len(lengths)))
        random.Random(seed).shuffle(order)
        self.T, self.n = [t for t, _ in lengths], [n for _, n in lengths]
        self.begin, rows = layout(lengths, order=order)
        self.N, self.H = sum(self.T), HK * G
        self.q = (1.5 * torch.randn((self.N, self.H, D), generator=gen)).to(DT[kind])
        used = torch.zeros(rows, dtype=torch.bool)
        for b, (_, n) in enumerate(lengths):
            used[self.begin[b]:self.begin[b] + n] = True
        self.cache = []
        for _ in range(2):
            self.cache.append(torch.randint(0, 256, (rows, HK, D // 2), generator=gen, dtype=torch.uint8))
            scales = torch.randint(powers[0], powers[1] + 1, (rows, HK, D // 32), generator=gen, dtype=torch.uint8)
            scales[~used] = 255
            self.cache.append(scales)
        self.q_layout, self.cache_layout = q_layout, cache_layout

    def values(self):
        return decode(*self.cache[:2]), decode(*self.cache[2:])

    def dev(self):
        t, off = self.torch, [0]
        for n in self.T:
            off.append(off[-1] + n)
        ints = lambda x, kind: t.tensor(x, dtype=kind, device="cuda")
        return dict(q=strided(self.q, self.q_layout), cache=tuple(strided(x, self.cache_layout) for x in self.cache),
                    offsets=ints(off, t.int32), kv_len=ints(self.n, t.int32), kv_begin=ints(self.begin, t.int64))

    def check(self, what, scale=0.0, max_q=None, **kw):
        import gated_delta_rule_varlen_amd as gdn

        out, lse = gdn.attention_fp4_varlen(**self.dev(), max_q=max(self.T) if max_q is None else max_q, scale=scale, return_lse=True,
                                            **kw)
        k, v = self.values()
        ref = attention_ref(self.q, k, v, self.T, self.begin, self.n, kind=self.kind, scale=scale or None)
        # fp32 queries and probabilities may be multiplied in three parts, each a sum of as many products
        by = 3.0 if self.kind == "f32" else 1.0
        # an exponential below fp32's normal range is zero: 2^-126 against a sum of at least one, for every key.  It shows
        # where the values of all other keys are zeros, as a sixteenth of the codes are.
        lost = 2.0 ** -126 * max(self.n) * v.nan_to_num().abs().max()
        assert_within(out, ref[0], by * ref[2] + lost, what + " out")
        assert_within(lse, ref[1], by * ref[3], what + " lse")
        return out, lse


TOKENS = [(1, 1), (1, 0), (0, 5), (1, 31), (1, 32), (1, 33), (1, 127), (1, 128), (1, 129), (1, 300), (0, 0), (1, 1000)]
BLOCKS = [(5, 300), (3, 2), (1, 0), (0, 9), (4, 4), (2, 33), (5, 129), (1, 64), (3, 1)]
PROMPTS = [(70, 70), (0, 11), (33, 200), (130, 130), (1, 5), (40, 3), (260, 517), (0, 0)]


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D", [32, 64, 96, 128, 160, 192, 224, 256])
def test_tokens(torch, kind, D):
    for HK, G in ((2, 4), (1, 1)):
        Case(torch, kind, HK, G, D, TOKENS).check(f"tokens {kind} {HK}x{G}x{D}")


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D", [32, 64, 128, 192, 256])
@pytest.mark.parametrize("G", [1, 3, 4, 5, 8, 12])
def test_blocks(torch, kind, D, G):
    """Up to 60 rows a sequence: one to four tiles of 16."""
    Case(torch, kind, 2, G, D, BLOCKS, cache_layout="rows").check(f"blocks {kind} {G}x{D}")


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("G,most", [(8, 8), (8, 5), (4, 16), (5, 9), (9, 7), (3, 21), (1, 40), (1, 64), (8, 9), (12, 9), (2, 50), (16, 32)])
def test_heads_divided_among_blocks(torch, kind, G, most):
    """Wide rows: a key head's query heads in one block, in several, and where they cannot be divided."""
    lengths = [(most, 200), (1, 1), (most - 1, 40), (2, 900), (0, 3)]
    c = Case(torch, kind, 2, G, 160, lengths)
    c.check(f"{kind} {most} x {G}")
    c.cache[3][c.begin[0] + 199, 1, 2] = 255  # and a value without a number in the last row
    import gated_delta_rule_varlen_amd as gdn

    out = torch.isnan(gdn.attention_fp4_varlen(**c.dev(), max_q=most)[0].cpu())
    assert out[most - 1, G:, 64:96].all() and out.sum() == 32 * G


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("D", [32, 64, 96, 128, 160, 256])
def test_prompts(torch, kind, D):
    Case(torch, kind, 2, 2, D, PROMPTS).check(f"prompts {kind} {D}")
    Case(torch, kind, 1, 5, D, PROMPTS[:4], cache_layout="wide", q_layout="wide").check(f"prompts {kind} {D}, 5 heads")


@pytest.mark.parametrize("cache_layout", ["rows", "heads", "wide"])
@pytest.mark.parametrize("q_layout", ["rows", "heads", "wide"])
def test_layouts(torch, cache_layout, q_layout):
    for lengths in (TOKENS, BLOCKS, PROMPTS):
        Case(torch, "bf16", 3, 2, 96, lengths, cache_layout, q_layout=q_layout).check(f"layout {cache_layout} {q_layout}")


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("max_q", [1, 7, 16, 17, 100, 10000])
def test_max_q_larger_than_the_longest(torch, kind, max_q):
    """The forms for one to many rows give the same rows."""
    Case(torch, kind, 2, 4, 64, TOKENS).check(f"max_q {max_q}", max_q=max_q)


@pytest.mark.parametrize("scale", [-0.2, 1.0, 1e-3])
def test_scales(torch, scale):
    for lengths in (TOKENS, BLOCKS, PROMPTS):
        Case(torch, "bf16", 2, 4, 128, lengths).check(f"scale {scale}", scale=scale)
        Case(torch, "f32", 2, 4, 64, lengths).check(f"scale {scale} f32", scale=scale)


@pytest.mark.parametrize("kind,powers", [("bf16", (60, 64)), ("bf16", (140, 146)), ("f16", (104, 110)), ("f16", (136, 140)),
                                         ("f32", (60, 64)), ("f32", (140, 146))])
def test_powers_far_out(torch, kind, powers):
    """Small and large values; with large ones a row attends to a single key."""
    c = Case(torch, kind, 2, 4, 64, TOKENS + BLOCKS, powers=powers)
    c.check(f"powers {powers}")


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("HK,G,D,n", [(1, 8, 256, 70000), (2, 1, 64, 33333), (8, 4, 128, 5001)])
def test_long_caches(torch, kind, HK, G, D, n):
    Case(torch, kind, HK, G, D, [(1, n)]).check(f"long {kind} {n}")
    Case(torch, kind, HK, G, D, [(3, n // 3), (0, 50), (1, 70), (2, n // 2)], cache_layout="rows").check(f"drafts {kind} {n}")


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_few_prompt_rows_over_a_long_cache(torch, kind):
    Case(torch, kind, 1, 4, 128, [(40, 20000), (33, 100)]).check(f"continued {kind}")
    Case(torch, kind, 2, 16, 64, [(30, 9000)], cache_layout="rows").check(f"continued {kind}, 16 heads")


def test_many_sequences(torch):
    rng = random.Random(4)
    Case(torch, "bf16", 2, 4, 64, [(rng.randint(0, 1), rng.randint(0, 90)) for _ in range(700)]).check("700 sequences")
    Case(torch, "f16", 1, 4, 64, [(rng.randint(0, 40), rng.randint(0, 90)) for _ in range(150)]).check("150 prompts")


def test_out_may_be_q_and_buffers_are_kept(torch):
    import gated_delta_rule_varlen_amd as gdn

    for lengths in (TOKENS, BLOCKS, PROMPTS):
        c = Case(torch, "bf16", 2, 4, 128, lengths)
        out, lse = c.check("apart")
        x = c.dev()
        ws = torch.empty(gdn.attention_fp4_workspace_bytes(x["q"], len(lengths), HK=2, max_q=max(c.T), kv_rows=len(c.cache[0])) + 16,
                         dtype=torch.uint8, device="cuda")
        stats = torch.empty_like(lse)
        y, z = gdn.attention_fp4_varlen(**x, max_q=max(c.T), out=x["q"], lse=stats, workspace=ws)
        assert y is x["q"] and z is stats
        assert (bits(y) == bits(out)).all() and (bits(z) == bits(lse)).all()
        assert gdn.attention_fp4_varlen(**c.dev(), max_q=max(c.T))[1] is None


def test_same_bits_again(torch):
    for lengths in ([(1, 9000), (1, 77)], BLOCKS, PROMPTS):
        c = Case(torch, "bf16", 2, 4, 128, lengths)
        first = c.check("once")
        for _ in range(2):
            again = c.check("again")
            assert all((bits(a) == bits(b)).all() for a, b in zip(first, again))


def check_without_numbers(torch, c, G, which):
    clean = c.check("clean")
    scales = c.cache[1 if which == "keys" else 3]
    for b, n in enumerate(c.n):
        scales[c.begin[b] + n - 1, 0, 1] = 255
    import gated_delta_rule_varlen_amd as gdn

    for where in ("apart", "q"):
        x = c.dev()
        out, lse = gdn.attention_fp4_varlen(**x, max_q=max(c.T), return_lse=True, out=x["q"] if where == "q" else None)
        last = torch.zeros(c.N, dtype=torch.bool)
        end = 0
        for t in c.T:
            end += t
            last[end - 1] = True
        hit = torch.isnan(out.cpu().float())
        assert not hit[~last].any() and not hit[:, G:].any(), "tokens that do not see the row, and the other head"
        if which == "keys":
            assert hit[last, :G].all() and torch.isnan(lse.cpu()[last, :G]).all()
        else:
            assert hit[last, :G, 32:64].all() and not hit[:, :, :32].any() and not hit[:, :, 64:].any() and not torch.isnan(lse).any()
        # the other rows have what they had, to the bound between two sums of the same terms
        k, v = c.values()
        k, v = torch.nan_to_num(k), torch.nan_to_num(v)
        ref = attention_ref(c.q, k, v, c.T, c.begin, c.n, kind=c.kind)
        by = 3.0 if c.kind == "f32" else 1.0
        for rows, heads in ((~last, slice(0, G)), (slice(None), slice(G, 2 * G))):
            assert_within(out[:, heads][rows], ref[0][:, heads][rows], by * ref[2][:, heads][rows], f"{which} out")
            assert_within(lse[:, heads][rows], ref[1][:, heads][rows], by * ref[3][:, heads][rows], f"{which} lse")
    assert not torch.isnan(clean[0]).any()


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("which", ["keys", "values"])
@pytest.mark.parametrize("lengths", [[(4, 40), (4, 300)], [(70, 170)], [(9, 200), (1, 5)]])
def test_blocks_without_numbers(torch, kind, which, lengths):
    """A scale byte of 255 in the last row of each sequence: only the last token may see it."""
    check_without_numbers(torch, Case(torch, kind, 2, 4, 64, lengths), 4, which)


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("which", ["keys", "values"])
@pytest.mark.parametrize("D,G,lengths", [(128, 4, [(4, 40), (4, 300)]), (128, 8, [(5, 3000), (2, 40)]), (256, 8, [(5, 4000), (2, 40)]),
                                         (192, 8, [(9, 400), (2, 30)]), (128, 4, [(90, 300)]), (256, 4, [(90, 300), (40, 70)])])
def test_blocks_without_numbers_in_wide_rows(torch, kind, which, D, G, lengths):
    """The same where row tiles share a block, where heads are divided among blocks, and in prompts."""
    check_without_numbers(torch, Case(torch, kind, 2, G, D, lengths), G, which)


def test_cache_of_no_rows_and_no_tokens(torch):
    import gated_delta_rule_varlen_amd as gdn

    cache = gdn.fp4_cache(0, 2, 64)
    q = torch.randn(3, 4, 64, device="cuda", dtype=torch.bfloat16)
    ints = lambda x, t=torch.int32: torch.tensor(x, dtype=t, device="cuda")
    at = dict(kv_len=ints([0, 0]), kv_begin=ints([0, 0], torch.int64))
    out, lse = gdn.attention_fp4_varlen(q, cache, ints([0, 1, 3]), return_lse=True, **at)
    assert (out == 0).all() and (lse == -math.inf).all()
    status = ints([5])
    out, _ = gdn.attention_fp4_varlen(q[:0], cache, ints([0, 0, 0]), dev_status=status, **at)
    assert out.shape == (0, 4, 64) and status.item() == 0


@pytest.mark.parametrize("lengths", [[(1, 40), (1, 9)], [(1, 4000), (1, 9)], [(60, 300), (40, 40)]])
@pytest.mark.parametrize("bad", ["first", "last", "falls", "max_q", "len", "begin", "end"])
def test_malformed_calls_write_nothing(torch, bad, lengths):
    import gated_delta_rule_varlen_amd as gdn

    c = Case(torch, "bf16", 2, 4, 64, lengths)
    x = c.dev()
    out, lse = sentinel((c.N, c.H, 64), "bf16"), sentinel((c.N, c.H), "f32")
    before = bits(out).copy(), bits(lse).copy()
    max_q = max(c.T)
    if bad == "first":
        x["offsets"][0] = 1
    elif bad == "last":
        x["offsets"][2] += 1
    elif bad == "falls":
        x["offsets"][1] = x["offsets"][2] + 1
    elif bad == "max_q":
        x["offsets"][1] = x["offsets"][2] if max_q == 1 else x["offsets"][1]
        max_q = 1 if max_q == 1 else max_q - 1
    elif bad == "len":
        x["kv_len"][1] = -1
    elif bad == "begin":
        x["kv_begin"][0] = -1
    else:
        x["kv_begin"][0] = len(c.cache[0]) - c.n[0] + 1
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    gdn.attention_fp4_varlen(**x, max_q=max_q, out=out, lse=lse, dev_status=status)
    assert status.item() == -9
    assert (bits(out) == before[0]).all() and (bits(lse) == before[1]).all()


@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("lengths", [[(1, 3000), (1, 1), (1, 77)], [(5, 900), (2, 60)], [(25, 900), (2, 60)], [(90, 400), (3, 3)]])
def test_streams_and_graphs(torch, lengths, D):
    """Two graphs with a workspace each, replayed in turn; another stream; lengths that change between replays."""
    import gated_delta_rule_varlen_amd as gdn

    cases = [Case(torch, "bf16", 2, 4, D, lengths, seed=s) for s in (1, 2)]
    runs = []
    for c in cases:
        out, lse = c.check("eager")
        x = c.dev()
        y, z = torch.empty_like(out), torch.empty_like(lse)
        ws = torch.empty(gdn.attention_fp4_workspace_bytes(x["q"], len(lengths), HK=2, max_q=max(c.T), kv_rows=len(c.cache[0])),
                         dtype=torch.uint8, device="cuda")
        call = lambda x=x, y=y, z=z, ws=ws, c=c: gdn.attention_fp4_varlen(**x, max_q=max(c.T), out=y, lse=z, workspace=ws)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            call()
        side.synchronize()
        assert (bits(y) == bits(out)).all()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        runs.append((graph, x, y, z, out, lse, (c, ws)))  # the graph needs its workspace
    for _ in range(3):
        for graph, x, y, z, out, lse, _ in runs:
            y.fill_(7.0)
            z.fill_(7.0)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert (bits(y) == bits(out)).all() and (bits(z) == bits(lse)).all()
    for graph, x, y, z, _, _, (c, _) in runs:  # fewer keys in the same buffers
        c.n = [max(n // 2, 1) for n in c.n]
        x["kv_len"].copy_(torch.tensor(c.n, dtype=torch.int32))
        want = c.check("fewer keys")
        graph.replay()
        torch.cuda.synchronize()
        assert (bits(y) == bits(want[0])).all() and (bits(z) == bits(want[1])).all()


def test_cache_past_32_bits(torch):
    """Runs at the end of a cache whose codes pass 2^32 bytes."""
    import gated_delta_rule_varlen_amd as gdn

    HK, D, rows = 2, 256, (1 << 32) // 256 + 1000
    cache = gdn.fp4_cache(rows, HK, D)
    for lengths in ([(1, 300), (1, 40)], [(80, 300)]):
        c = Case(torch, "bf16", HK, 2, D, lengths)
        x = c.dev()
        at = rows - len(c.cache[0])
        for big, part in zip(cache, x["cache"]):
            big[at:] = part
        x["cache"], x["kv_begin"] = cache, x["kv_begin"] + at
        out, _ = gdn.attention_fp4_varlen(**x, max_q=max(c.T))
        k, v = c.values()
        ref = attention_ref(c.q, k, v, c.T, c.begin, c.n, kind="bf16")
        assert_within(out, ref[0], ref[2], f"far rows {lengths}")

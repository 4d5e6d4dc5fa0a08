"""GPU tests of gdn_attention_varlen and gdn_attention_prefix_varlen against a plain 64-bit attention:
types, head widths and layouts, lengths around every tile edge, rows without keys, values in places
that are masked, long runs cut in parts, malformed calls, streams and graphs."""
import random

import pytest

from attn_util import DT, assert_within, attention_ref, layout
from gpu_util import bits, ensure_built, require_gpu, sentinel

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    ensure_built()
    return require_gpu()


class Case:
    """Seeded inputs on the CPU and the device: lengths are (new tokens, cache rows) per sequence."""

    def __init__(self, torch, kind, HK, G, D, lengths, prefix=0, heads_major=False, seed=1, padded_q=False):
        self.torch, self.kind, self.lengths = torch, kind, lengths
        gen = torch.Generator().manual_seed(seed)
        order = list(range(len(lengths)))
        random.Random(seed).shuffle(order)
        self.T, self.n = [t for t, _ in lengths], [n for _, n in lengths]
        self.begin, rows = layout(lengths, order=order)
        self.N, self.H = sum(self.T), HK * G

        def normal(*shape, scale=1.0):
            return (scale * torch.randn(shape, generator=gen)).to(DT[kind])

        self.q = normal(self.N, self.H, D, scale=1.5)
        self.kv = [normal(HK, rows, D).permute(1, 0, 2) if heads_major else normal(rows, HK, D) for _ in range(2)]
        # rows of no sequence hold NaN
        used = torch.zeros(rows, dtype=torch.bool)
        for b, (_, n) in enumerate(lengths):
            used[self.begin[b]:self.begin[b] + n] = True
        for x in self.kv:
            x[~used] = float("nan")
        self.prefix = [normal(prefix, HK, D) for _ in range(2)] if prefix else None
        self.padded_q = padded_q

    def dev(self):
        t, dev = self.torch, "cuda"

        def move(x):  # keeps the strides
            return x.permute(1, 0, 2).contiguous().to(dev).permute(1, 0, 2) if not x.is_contiguous() else x.to(dev)

        off = [0]
        for n in self.T:
            off.append(off[-1] + n)
        q = self.q.to(dev)
        if self.padded_q:  # a part of a wider row
            wide = t.full((self.N, self.H + 3, self.q.shape[2]), float("nan"), dtype=q.dtype, device=dev)
            wide[:, 1:1 + self.H] = q
            q = wide[:, 1:1 + self.H]
        return dict(q=q, k=move(self.kv[0]), v=move(self.kv[1]), offsets=t.tensor(off, dtype=t.int32, device=dev),
                    kv_begin=t.tensor(self.begin, dtype=t.int64, device=dev),
                    kv_len=t.tensor(self.n, dtype=t.int32, device=dev), max_q=max(self.T + [1]), return_lse=True)

    def call(self, x=None, **kw):
        import gated_delta_rule_varlen_amd as gdn

        x = {**(x or self.dev()), **kw}
        q, k, v, off = (x.pop(n) for n in ("q", "k", "v", "offsets"))
        if self.prefix is None:
            return gdn.attention_varlen(q, k, v, off, **x)
        return gdn.attention_prefix_varlen(q, *(p.cuda() for p in self.prefix), k, v, off, **x)

    def ref(self, **kw):
        p = self.prefix or (None, None)
        return attention_ref(self.q, *self.kv, self.T, self.begin, self.n, kind=self.kind, prefix_k=p[0], prefix_v=p[1],
                             **kw)

    def check(self, what):
        print(f"[case] {what} {self.kind} q {tuple(self.q.shape)} HK {self.kv[0].shape[1]} lengths {self.lengths[:12]}",
              flush=True)
        out, lse = self.call()
        self.torch.cuda.synchronize()
        o, l, o_tol, l_tol = self.ref()
        assert out.dtype == DT[self.kind] and lse.dtype == self.torch.float32
        assert_within(out, o, o_tol, what + " out")
        assert_within(lse, l, l_tol, what + " lse")


KINDS = ["bf16", "f16", "f32"]
# new tokens and cache rows around the edges of 32-, 64-, 128- and 256-key tiles, empty ones among them
DECODE = [(1, n) for n in (1, 2, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 300)] + [(0, 7), (0, 0), (1, 515)]
BLOCKS = [(4, 4), (5, 36), (1, 1), (0, 0), (9, 200), (2, 130), (7, 64), (3, 65), (6, 512)]
PROMPTS = [(130, 130), (1, 1), (0, 0), (64, 64), (65, 65), (300, 300), (31, 95), (33, 161), (128, 500)]
NO_KEYS = [(3, 0), (4, 2), (1, 0), (40, 7), (1, 9), (2, 2), (0, 3)]
SETS = {"decode": DECODE, "blocks": BLOCKS, "prompts": PROMPTS, "no_keys": NO_KEYS}


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("HK,G,D", [(2, 4, 64), (2, 4, 128), (1, 8, 256), (2, 2, 32), (1, 3, 96), (3, 1, 72), (1, 5, 80),
                                    (1, 16, 192), (2, 1, 8)])
@pytest.mark.parametrize("name", SETS)
def test_lengths_types_and_widths(torch, kind, HK, G, D, name):
    Case(torch, kind, HK, G, D, SETS[name], seed=D + G).check(f"{name} D{D}")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("HK,G,D,prefix", [(2, 4, 64, 1001), (2, 4, 128, 1), (1, 8, 256, 130), (1, 3, 72, 64), (1, 16, 96, 700)])
@pytest.mark.parametrize("name", ["decode", "blocks", "prompts", "no_keys"])
def test_shared_prefix(torch, kind, HK, G, D, prefix, name):
    Case(torch, kind, HK, G, D, SETS[name], prefix=prefix, seed=prefix).check(f"prefix {prefix} {name} D{D}")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("HK,G,D,lengths", [
    (1, 4, 64, [(1, 5000)]),            # one sequence: its keys are cut in parts
    (2, 8, 256, [(5, 3333), (2, 40)]),
    (1, 2, 128, [(300, 4000)]),         # several row tiles over a long cache
    (4, 16, 64, [(9, 700), (1, 900)]),  # more rows than one tile in a short call
    (1, 1, 128, [(1, 64 * i + 3) for i in range(70)]),
    (2, 1, 32, [(1, 1)] * 300),         # more sequences than a block has threads
    (1, 7, 64, [(700, 700), (5, 1500)]),
])
def test_long_and_many(torch, kind, HK, G, D, lengths):
    Case(torch, kind, HK, G, D, lengths, seed=5).check("long")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("prefix", [0, 77])
def test_layouts(torch, kind, prefix):
    """Heads-major caches and queries that are part of a wider row give the bits of the plain layout."""
    for lengths in (DECODE, PROMPTS):
        same = []
        for heads_major in (False, True):
            c = Case(torch, kind, 2, 4, 64, lengths, prefix=prefix, seed=3)
            if heads_major:
                c.kv = [x.permute(1, 0, 2).contiguous().permute(1, 0, 2) for x in c.kv]
                c.padded_q = True
            same.append(c.call())
        torch.cuda.synchronize()
        for a, b in zip(*same):
            assert (bits(a) == bits(b)).all()


@pytest.mark.parametrize("kind", KINDS)
def test_packed_keys(torch, kind):
    """Without kv_begin and kv_len the keys are packed like the queries."""
    import gated_delta_rule_varlen_amd as gdn

    T = [5, 0, 130, 1, 64]
    gen = torch.Generator().manual_seed(9)
    q, k, v = (torch.randn((sum(T), h, 64), generator=gen).to(DT[kind]) for h in (8, 2, 2))
    off = [0, 5, 5, 135, 136, 200]
    out, lse = gdn.attention_varlen(q.cuda(), k.cuda(), v.cuda(), torch.tensor(off, dtype=torch.int32).cuda(),
                                    return_lse=True)
    o, l, ot, lt = attention_ref(q, k, v, T, off, T, kind=kind)
    assert_within(out, o, ot, "packed out")
    assert_within(lse, l, lt, "packed lse")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("HK,G,D,lengths,prefix", [
    (1, 4, 64, [(6, 40), (3, 3)], 0),
    (2, 2, 128, [(70, 170), (200, 200)], 0),
    (1, 4, 256, [(40, 40)], 33),
])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_masked_rows_hold_anything(torch, kind, HK, G, D, lengths, prefix, value):
    """The last token's key and value reach no earlier token, even where they are not finite."""
    c = Case(torch, kind, HK, G, D, lengths, prefix=prefix, seed=8)
    for b, (_, n) in enumerate(lengths):
        for x in c.kv:
            x[c.begin[b] + n - 1] = value
    out, lse = c.call()
    o, l, ot, lt = c.ref()
    keep = torch.ones(c.N, dtype=torch.bool)
    end = 0
    for t in c.T:
        end += t
        keep[end - 1] = False
    assert_within(out[keep.cuda()], o[keep], ot[keep], "masked out")
    assert_within(lse[keep.cuda()], l[keep], lt[keep], "masked lse")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lengths", [[(1, 900), (1, 3)], [(5, 300)], [(150, 400)]])
def test_sharp_and_growing_scores(torch, kind, lengths):
    """Scores that span hundreds and grow along the keys: the running maximum moves at every tile."""
    c = Case(torch, kind, 1, 4, 64, lengths, seed=12)
    for b, (_, n) in enumerate(lengths):
        ramp = torch.linspace(0.2, 6.0, n)[:, None, None]
        rows = slice(c.begin[b], c.begin[b] + n)
        c.kv[0][rows] = (c.kv[0][rows].float() * ramp + ramp).to(DT[kind])
    c.q = (c.q.float() * 2 + 1).to(DT[kind])
    c.check("growing")


@pytest.mark.parametrize("scale", [0.0, 0.03, -0.2])
def test_scale(torch, scale):
    c = Case(torch, "f32", 2, 2, 64, [(3, 50), (70, 90), (1, 200)], seed=14)
    out, lse = c.call(scale=scale)
    o, l, ot, lt = c.ref(scale=scale or None)
    assert_within(out, o, ot, "scaled out")
    assert_within(lse, l, lt, "scaled lse")


def _expect_untouched(torch, c, status=-9, **kw):
    x = c.dev()
    out, lse = sentinel((c.N, c.H, c.q.shape[2]), c.kind), sentinel((c.N, c.H), "f32")
    want = bits(out).copy(), bits(lse).copy()
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    for name, at, value in kw.pop("spoil", ()):
        x[name][at] = value
    c.call(x, out=out, lse=lse, dev_status=st, **kw)
    torch.cuda.synchronize()
    assert st.item() == status
    assert ((bits(out) == want[0]).all() and (bits(lse) == want[1]).all()) == (status != 0)


@pytest.mark.parametrize("prefix", [0, 40])
@pytest.mark.parametrize("lengths", [[(1, 70), (1, 5), (1, 300)], [(100, 150), (0, 4), (230, 260)]])
@pytest.mark.parametrize("what", ["ok", "start", "end", "falling", "longest", "begin", "run", "far", "length"])
def test_malformed_calls_write_nothing(torch, lengths, prefix, what):
    c = Case(torch, "bf16", 2, 4, 64, lengths, prefix=prefix, seed=2)
    rows = c.kv[0].shape[0]
    spoil = dict(ok=[], start=[("offsets", 0, 1)], end=[("offsets", 3, c.N + 1)], falling=[("offsets", 1, c.N + 5)],
                 longest=[], begin=[("kv_begin", 1, -1)], run=[("kv_begin", 2, rows - c.n[2] + 1)],
                 far=[("kv_begin", 0, 1 << 62)], length=[("kv_len", 0, -1)])[what]
    kw = dict(max_q=max(c.T) - 1) if what == "longest" else {}
    if what == "longest" and max(c.T) == 1:
        pytest.skip("max_q 0 is refused on the host")
    _expect_untouched(torch, c, status=0 if what == "ok" else -9, spoil=spoil, **kw)


def test_calls_without_tokens(torch):
    c = Case(torch, "bf16", 2, 2, 64, [(0, 5), (0, 0)], seed=2)
    st = torch.ones(1, dtype=torch.int32, device="cuda")
    out, lse = c.call(dev_status=st)
    torch.cuda.synchronize()
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4) and st.item() == 0


def test_binding_refuses_what_it_cannot_describe(torch):
    c = Case(torch, "bf16", 2, 4, 64, [(1, 9), (2, 5)], seed=2)
    x = c.dev()
    half = x["k"].half()
    for bad, err in ((dict(k=half), TypeError), (dict(k=x["k"][:, :, :32]), ValueError), (dict(k=x["k"][:5]), ValueError),
                     (dict(kv_len=x["kv_len"].long()), TypeError), (dict(kv_begin=x["kv_begin"][:1]), ValueError),
                     (dict(offsets=x["offsets"].cpu()), ValueError), (dict(v=x["v"].cpu()), ValueError),
                     (dict(q=x["q"].transpose(1, 2)), ValueError), (dict(lse=x["kv_begin"]), TypeError),
                     (dict(out=x["q"][:2]), ValueError)):
        with pytest.raises(err):
            c.call({**x, **bad})


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_offsets_past_32_bits(torch, kind):
    """A run at the end of a cache of more than 2^32 bytes and 2^31 elements."""
    import gated_delta_rule_varlen_amd as gdn

    HK, D, n = 4, 64, 700
    rows = (1 << 31) // (HK * D) + 300  # the run starts below element 2^31 and ends past it
    gen = torch.Generator().manual_seed(4)
    q = torch.randn((3, 8, D), generator=gen).to(DT[kind])
    k, v = (torch.randn((n, HK, D), generator=gen).to(DT[kind]) for _ in range(2))
    cache = [torch.empty((rows, HK, D), dtype=DT[kind], device="cuda") for _ in range(2)]
    for c, x in zip(cache, (k, v)):
        c[rows - n:] = x.cuda()
    out, lse = gdn.attention_varlen(q.cuda(), *cache, torch.tensor([0, 3], dtype=torch.int32).cuda(),
                                    kv_begin=torch.tensor([rows - n]).cuda(),
                                    kv_len=torch.tensor([n], dtype=torch.int32).cuda(), max_q=3, return_lse=True)
    o, l, ot, lt = attention_ref(q, k, v, [3], [0], [n], kind=kind)
    assert_within(out, o, ot, "far out")
    assert_within(lse, l, lt, "far lse")


@pytest.mark.parametrize("prefix", [0, 500])
@pytest.mark.parametrize("lengths", [[(1, 3000), (1, 40)], [(200, 900), (3, 70)]])
def test_repeats_streams_and_graphs(torch, prefix, lengths):
    """The same bits on a second run, on another stream, and from replays of a captured graph whose
    inputs change between them."""
    c = Case(torch, "bf16", 2, 4, 128, lengths, prefix=prefix, seed=6)
    x = c.dev()
    first = c.call(x)
    pre = [p.cuda() for p in c.prefix] if prefix else None
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(other):
        second = c.call(x)
    torch.cuda.synchronize()
    for a, b in zip(first, second):
        assert (bits(a) == bits(b)).all()

    import gated_delta_rule_varlen_amd as gdn

    out, lse = torch.empty_like(first[0]), torch.empty_like(first[1])
    args = [x["q"]] + (pre or []) + [x["k"], x["v"], x["offsets"]]
    kw = {n: x[n] for n in ("kv_begin", "kv_len", "max_q")}
    f = gdn.attention_prefix_varlen if prefix else gdn.attention_varlen
    need = gdn.attention_workspace_bytes(x["q"], len(lengths), HK=2, max_q=kw["max_q"], kv_rows=len(x["k"]), prefix_len=prefix)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f(*args, **kw, out=out, lse=lse, workspace=ws)
    for turn in range(4):
        x["q"].copy_(c.q.cuda() * (1 + turn))
        want = f(*args, **kw, return_lse=True)
        torch.cuda.synchronize()
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert (bits(out) == bits(want[0])).all() and (bits(lse) == bits(want[1])).all(), turn


@pytest.mark.parametrize("seed", range(24))
def test_random_shapes(torch, seed):
    r = random.Random(1000 + seed)
    kind = r.choice(KINDS)
    HK, G = r.choice([1, 2, 3, 4]), r.choice([1, 2, 3, 4, 5, 8, 16])
    D = r.choice([32, 64, 72, 80, 96, 128, 192, 256])
    longest = r.choice([1, 2, 9, 60, 400])
    B = r.randrange(1, 12)
    lengths = []
    for _ in range(B):
        t = r.randrange(0, longest + 1)
        lengths.append((t, max(0, t + r.choice([0, 0, -2, r.randrange(700)]))))
    if sum(t for t, _ in lengths) == 0:
        lengths[0] = (1, 5)
    Case(torch, kind, HK, G, D, lengths, prefix=r.choice([0, 0, r.randrange(1, 600)]), seed=seed).check(f"random {seed}")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("G,D,lengths,prefix", [
    (4, 64, [(6, 40), (3, 3)], 0),       # short form, runs whole in a block and cut
    (2, 128, [(70, 170), (200, 200)], 0),  # long form
    (4, 256, [(40, 40)], 33),
    (1, 64, [(5, 90), (1, 20)], 70),
])
@pytest.mark.parametrize("value", [0.5, float("nan"), float("inf")])
def test_out_may_be_the_queries(torch, kind, G, D, lengths, prefix, value):
    """out = q gives the bits of an output of its own, where masked values make rows be done again too."""
    c = Case(torch, kind, 2, G, D, lengths, prefix=prefix, seed=8, padded_q=True)
    for b, (_, n) in enumerate(lengths):
        for x in c.kv:
            x[c.begin[b] + n - 1] = value
    want, want_lse = c.call()
    x = c.dev()
    out, lse = c.call(x, out=x["q"])
    torch.cuda.synchronize()
    assert out.data_ptr() == x["q"].data_ptr()
    assert (bits(out) == bits(want)).all() and (bits(lse) == bits(want_lse)).all()


@pytest.mark.parametrize("max_q", [3, 0, -1, -1000])
def test_calls_without_tokens_take_any_max_q(torch, max_q):
    c = Case(torch, "bf16", 2, 2, 64, [(0, 5), (0, 0)], seed=2)
    st = torch.ones(1, dtype=torch.int32, device="cuda")
    c.call(dev_status=st, max_q=max_q)
    torch.cuda.synchronize()
    assert st.item() == 0


def test_more_rows_behind_a_prefix_than_one_axis_of_a_grid(torch):
    """2^26 rows and more joined with a prefix; sequences read the same rows of the cache."""
    import gated_delta_rule_varlen_amd as gdn

    H, D, T, n, P = 32, 8, 128, 130, 40
    B = (1 << 26) // (H * T) + 1
    gen = torch.Generator(device="cuda").manual_seed(5)
    normal = lambda *s: torch.randn(s, generator=gen, device="cuda", dtype=torch.bfloat16)
    q, k, v, pk, pv = normal(B * T, H, D), normal(n, H, D), normal(n, H, D), normal(P, H, D), normal(P, H, D)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    out, lse = gdn.attention_prefix_varlen(q, pk, pv, k, v, torch.arange(B + 1, device="cuda", dtype=torch.int32) * T,
                                           kv_len=i32([n] * B), kv_begin=torch.zeros(B, dtype=torch.int64, device="cuda"),
                                           max_q=T, return_lse=True)
    for b in (0, B // 2, B - 1):
        at = slice(b * T, (b + 1) * T)
        o, l, ot, lt = attention_ref(q[at].cpu(), k.cpu(), v.cpu(), [T], [0], [n], kind="bf16", prefix_k=pk.cpu(),
                                     prefix_v=pv.cpu())
        assert_within(out[at], o, ot, f"sequence {b} out")
        assert_within(lse[at], l, lt, f"sequence {b} lse")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("HK,G,D,lengths,prefix", [
    (2, 4, 64, [(i % 5 != 2, 1 + (37 * i) % 90) for i in range(300)], 0),  # single tokens
    (1, 3, 128, [(700, 900)] + [(i % 4, 3 + i % 60) for i in range(70)], 0),  # a token's rows in two tiles
    (1, 8, 256, [(i % 6, 2 + i % 7) for i in range(200)] + [(0, 0), (400, 450)], 77),
    (1, 2, 64, [(i % 3, 1 + i % 4) for i in range(5000)], 0),  # more than 64 * 64 sequences
])
def test_default_max_q(torch, kind, HK, G, D, lengths, prefix):
    c = Case(torch, kind, HK, G, D, lengths, prefix=prefix, seed=D)
    out, lse = c.call(max_q=None)
    o, l, ot, lt = c.ref()
    assert_within(out, o, ot, "default max_q out")
    assert_within(lse, l, lt, "default max_q lse")


def test_default_max_q_of_a_large_batch(torch):
    """8192 single tokens of 32 heads: as many row tiles for each as for a sequence of all tokens would pass the
    threads of one launch."""
    import gated_delta_rule_varlen_amd as gdn

    B, H, HK, D = 8192, 32, 8, 64
    gen = torch.Generator(device="cuda").manual_seed(3)
    normal = lambda *s: torch.randn(s, generator=gen, device="cuda").bfloat16()
    n = 1 + torch.arange(B) % 3
    begin = torch.nn.functional.pad(n.cumsum(0), (1, 0))
    q, k, v = normal(B, H, D), normal(int(begin[-1]), HK, D), normal(int(begin[-1]), HK, D)
    out, lse = gdn.attention_varlen(q, k, v, torch.arange(B + 1, dtype=torch.int32).cuda(), kv_len=n.int().cuda(),
                                    kv_begin=begin[:-1].cuda(), return_lse=True, out=sentinel((B, H, D), "bf16"))
    pick = [0, 1, 2, 63, 64, 127, 128, 4095, 4096, B - 2, B - 1]
    o, l, ot, lt = attention_ref(q[pick].cpu(), k.cpu(), v.cpu(), [1] * len(pick), begin[pick].tolist(), n[pick].tolist(),
                                 kind="bf16")
    assert_within(out[pick], o, ot, "large batch out")
    assert_within(lse[pick], l, lt, "large batch lse")
    assert torch.isfinite(out.float()).all() and torch.isfinite(lse).all()
    one = n == 1  # a token that sees one key has its value
    want = v[begin[:-1][one].cuda()].repeat_interleave(H // HK, dim=1)
    assert (bits(out[one.cuda()]) == bits(want)).all()


@pytest.mark.parametrize("what", ["ok", "start", "end", "falling", "far", "length"])
def test_default_max_q_malformed(torch, what):
    c = Case(torch, "bf16", 2, 4, 64, [(1 + i % 3, 20 + i) for i in range(150)], seed=2)
    spoil = dict(ok=[], start=[("offsets", 0, 1)], end=[("offsets", 150, c.N + 1)], falling=[("offsets", 70, 1 << 30)],
                 far=[("offsets", 64, -(1 << 31))], length=[("kv_len", 0, -1)])[what]
    _expect_untouched(torch, c, status=0 if what == "ok" else -9, spoil=spoil, max_q=None)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("HK,G,lengths,prefix", [
    (1, 8, [(300, 300)], 0),
    (2, 3, [(90, 90), (0, 5), (130, 400), (3, 0)], 0),  # a token's rows in two tiles
    (1, 4, [(150, 150), (60, 20)], 500),
])
def test_a_large_cache_is_not_cut_finer(torch, kind, HK, G, lengths, prefix):
    """Key parts are of the sequences' own keys, however many rows the cache has: no part of less than 128 keys
    is written to the workspace."""
    import gated_delta_rule_varlen_amd as gdn

    D = 64
    c = Case(torch, kind, HK, G, D, lengths, prefix=prefix, seed=21)
    x = c.dev()
    for n in ("k", "v"):
        large = torch.full((1 << 17, HK, D), float("nan"), dtype=DT[kind], device="cuda")
        large[:len(x[n])] = x[n]
        x[n] = large
    need = gdn.attention_workspace_bytes(x["q"], len(lengths), HK=HK, max_q=x["max_q"], kv_rows=1 << 17, prefix_len=prefix)
    ws = torch.full((need,), 0xA5, dtype=torch.uint8, device="cuda")
    out, lse = c.call(x, workspace=ws)
    torch.cuda.synchronize()
    parts = [max(1, (prefix + n) // 128) for _, n in lengths]
    most = sum(p * t for p, (t, _) in zip(parts, lengths)) * c.H * (D + 2) + c.N + 1
    written = (ws[:need // 4 * 4].view(torch.int32) != torch.tensor(0xA5A5A5A5 - (1 << 32), dtype=torch.int32, device="cuda")).sum().item()
    o, l, ot, lt = c.ref()
    assert_within(out, o, ot, "large cache out")
    assert_within(lse, l, lt, "large cache lse")
    assert written <= most, (written, most)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows", [16, 24, 32, 40, 48, 56, 64, 72, 128])
@pytest.mark.parametrize("prefix", [0, 90])
def test_rows_of_every_number_of_waves(torch, kind, D, rows, prefix):
    """Every number of waves (16 rows each) of the short form, at every width, whole runs and cut ones."""
    Case(torch, kind, 2, 8, D, [(rows // 8, 400), (1, 33), (0, 4), (rows // 8, rows // 8), (2, 1)], prefix=prefix,
         seed=rows + D).check(f"{rows} rows D{D}")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("T,B", [(1, 150), (5, 30)])
def test_many_rows_of_cut_runs(torch, kind, D, T, B):
    """More rows than are joined a block each: single tokens and drafts of 32 heads, empty sequences, rows without
    keys and a run over many blocks among them."""
    lengths = [(0 if i % 11 == 5 else T, (T - 2 if T > 2 and i % 13 == 7 else T + (37 * i) % 90)) for i in range(B)]
    lengths[B // 2] = (T, 3000)
    c = Case(torch, kind, 8, 4, D, lengths, seed=D + T)
    assert c.N * c.H > 2048
    c.check(f"cut runs D{D} T{T}")


@pytest.mark.parametrize("kind", KINDS)
def test_many_rows_of_cut_runs_masked_values(torch, kind):
    """The last token's value of every sequence is not finite; cut runs join rows done again and rows that are not."""
    c = Case(torch, kind, 8, 4, 64, [(5, 40 + 61 * i % 700) for i in range(20)], seed=3)
    last = torch.zeros(c.N, dtype=torch.bool)
    last[4::5] = True
    for b, (_, n) in enumerate(c.lengths):
        for x in c.kv:
            x[c.begin[b] + n - 1] = float("nan")
    out, lse = c.call()
    o, l, ot, lt = c.ref()
    assert_within(out[~last.cuda()], o[~last], ot[~last], "cut masked out")
    assert_within(lse[~last.cuda()], l[~last], lt[~last], "cut masked lse")


@pytest.mark.parametrize("what", ["ok", "falling", "run", "length"])
def test_many_rows_malformed(torch, what):
    c = Case(torch, "bf16", 8, 4, 64, [(1, 20 + i) for i in range(100)], seed=2)
    rows = c.kv[0].shape[0]
    spoil = dict(ok=[], falling=[("offsets", 1, c.N + 5)], run=[("kv_begin", 2, rows - c.n[2] + 1)],
                 length=[("kv_len", 0, -1)])[what]
    _expect_untouched(torch, c, status=0 if what == "ok" else -9, spoil=spoil)


def test_many_rows_from_a_graph(torch):
    """Replays whose lengths change between them: other runs are cut than when the call was captured."""
    import gated_delta_rule_varlen_amd as gdn

    c = Case(torch, "bf16", 8, 4, 128, [(1, 60 + 13 * i % 200) for i in range(100)], seed=6)
    x = c.dev()
    kw = {n: x[n] for n in ("kv_begin", "kv_len", "max_q")}
    args = [x[n] for n in ("q", "k", "v", "offsets")]
    out, lse = (torch.empty_like(t) for t in gdn.attention_varlen(*args, **kw, return_lse=True))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.attention_varlen(*args, **kw, out=out, lse=lse)
    for turn in range(4):
        x["kv_len"].copy_(torch.tensor([max(1, n - turn * (i % 3) * 20) for i, n in enumerate(c.n)], dtype=torch.int32))
        want = gdn.attention_varlen(*args, **kw, return_lse=True)
        torch.cuda.synchronize()
        out.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert (bits(out) == bits(want[0])).all() and (bits(lse) == bits(want[1])).all(), turn


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("lengths", [[(3, 50), (1, 200)], [(70, 90), (3, 50)]])
def test_negative_scale(torch, kind, lengths):
    c = Case(torch, kind, 2, 4, 128, lengths, seed=14)
    out, lse = c.call(scale=-0.2)
    o, l, ot, lt = c.ref(scale=-0.2)
    assert_within(out, o, ot, "scaled out")
    assert_within(lse, l, lt, "scaled lse")


@pytest.mark.parametrize("T", [[3, 1], [200, 5]])
def test_a_cache_without_rows(torch, T):
    """No keys anywhere: zeros and -inf; and a prefix without rows is no prefix."""
    import gated_delta_rule_varlen_amd as gdn

    N, dev = sum(T), "cuda"
    q = torch.randn(N, 4, 64, device=dev, dtype=torch.bfloat16)
    none = torch.empty(0, 2, 64, device=dev, dtype=torch.bfloat16)
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=dev)
    kw = dict(kv_begin=torch.zeros(2, dtype=torch.int64, device=dev), max_q=max(T), return_lse=True)
    off = i32(0, T[0], N)
    out, lse = gdn.attention_varlen(q, none, none, off, kv_len=i32(0, 0), **kw)
    assert (out == 0).all() and (lse == -float("inf")).all()
    k, v = (torch.randn(9, 2, 64, device=dev, dtype=torch.bfloat16) for _ in range(2))
    want = gdn.attention_varlen(q, k, v, off, kv_len=i32(4, 9), **kw)
    got = gdn.attention_prefix_varlen(q, none, none, k, v, off, kv_len=i32(4, 9), **kw)
    for a, b in zip(got, want):
        assert (bits(a) == bits(b)).all()


def test_binding_names_what_it_refuses(torch):
    """With device tensors that are right otherwise: the number or tensor that is none is what the error names."""
    import gated_delta_rule_varlen_amd as gdn

    c = Case(torch, "bf16", 2, 4, 64, [(1, 9), (2, 5)], seed=2)
    x = c.dev()
    c.call(x)
    for bad, err, match in ((dict(k=3), TypeError, "k must be a tensor"), (dict(v="v"), TypeError, "v must be a tensor"),
                            (dict(offsets=3), TypeError, "offsets must be a tensor"),
                            (dict(q=None), TypeError, "q must be a tensor"),
                            (dict(out=3), TypeError, "out must be a tensor"),
                            (dict(workspace=3), TypeError, "workspace must be a tensor"),
                            (dict(scale="one"), TypeError, "real number"), (dict(max_q="one"), TypeError, "integer"),
                            (dict(max_q=1 << 70), OverflowError, "int too")):
        with pytest.raises(err, match=match):
            c.call({**x, **bad})
    k = torch.randn(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    rope = dict(inv_freq=torch.ones(32, device="cuda"))
    gdn.qk_norm_rope_varlen(x["q"], k, k, x["offsets"], **rope)
    for args, kw, match in (((x["q"], 3, k, x["offsets"]), {}, "k must be a tensor"),
                            ((x["q"], k, k, None), {}, "offsets must be a tensor"),
                            ((x["q"], k, k, x["offsets"]), dict(eps="small"), "real number"),
                            ((x["q"], k, k, x["offsets"]), dict(inv_freq=None), "inv_freq must be a tensor")):
        with pytest.raises(TypeError, match=match):
            gdn.qk_norm_rope_varlen(*args, **{**rope, **kw})


def test_binding_refuses_v_out_without_v(torch):
    import gated_delta_rule_varlen_amd as gdn

    k, off = torch.randn(3, 2, 64, device="cuda"), torch.tensor([0, 3], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="v_out without v"):
        gdn.qk_norm_rope_varlen(k, k, None, off, inv_freq=torch.ones(32, device="cuda"), v_out=torch.empty_like(k))


def test_binding_refuses_a_truth_value_that_has_none(torch):
    c = Case(torch, "bf16", 2, 4, 64, [(1, 9), (2, 5)], seed=2)
    with pytest.raises(RuntimeError, match="ambiguous"):
        c.call({**c.dev(), "return_lse": torch.ones(2)})


def test_binding_refuses_a_workspace_elsewhere(torch):
    c = Case(torch, "bf16", 2, 4, 64, [(1, 9), (2, 5)], seed=2)
    with pytest.raises(ValueError, match="workspace .* cuda:0"):
        c.call({**c.dev(), "workspace": torch.empty(1 << 20, dtype=torch.uint8)})


@pytest.mark.parametrize("D", [128, 256])
@pytest.mark.parametrize("at", [0, 37, 100, 127])
def test_scores_of_single_precision_are_sums_of_parts(torch, D, at):
    """One large product among many that a running sum behind it would lose: of single tokens at most a quarter of them
    may be.  With one key the lse is the score; e = 2^-24 of it is 1, and no more than eight roundings follow."""
    import gated_delta_rule_varlen_amd as gdn

    q = torch.full((3, 2, D), 0.5, device="cuda")
    q[:, :, at] = 4096.0
    one = torch.ones(3, dtype=torch.int32, device="cuda")
    _, lse = gdn.attention_varlen(q, q, q, torch.arange(4, dtype=torch.int32, device="cuda"), kv_len=one,
                                  kv_begin=torch.arange(3, device="cuda"), max_q=1, scale=1.0, return_lse=True)
    exact = 2.0 ** 24 + 0.25 * (D - 1)
    assert (lse.double() - exact).abs().max().item() <= 0.25 * D / 4 + 8

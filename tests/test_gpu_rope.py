"""GPU tests of gdn_qk_norm_rope_varlen against a plain 64-bit norm and rotation."""
import pytest

from attn_util import DT, assert_within, layout, rope_ref
from gpu_util import bits, ensure_built, require_gpu, sentinel

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    ensure_built()
    return require_gpu()


KINDS = ["bf16", "f16", "f32"]


class Case:
    def __init__(self, torch, kind, H, HK, D, rot, T, past, first=None, seed=1, heads_major=False, weights=True):
        self.torch, self.kind, self.T, self.past, self.rot = torch, kind, T, past, rot
        gen = torch.Generator().manual_seed(seed)
        self.N, self.H, self.HK, self.D = sum(T), H, HK, D
        self.row = torch.randn((self.N, (H + 2 * HK) * D), generator=gen).to(DT[kind])
        self.w = [1 + 0.2 * torch.randn(D, generator=gen) if weights else None for _ in range(2)]
        self.inv_freq = (1e6 ** (-torch.arange(0, rot, 2).double() / max(rot, 1))).float()
        self.begin, self.rows = layout([(t, p + t) for t, p in zip(T, past)], order=list(range(len(T)))[::-1])
        self.first = past if first is None else first
        self.heads_major = heads_major
        self.off = [0]
        for t in T:
            self.off.append(self.off[-1] + t)

    def parts(self, row):
        H, HK, D, N = self.H, self.HK, self.D, self.N
        return (row[:, :H * D].view(N, H, D), row[:, H * D:(H + HK) * D].view(N, HK, D),
                row[:, (H + HK) * D:].view(N, HK, D))

    def dev(self):
        t = self.torch
        caches = []
        for _ in range(2):
            if self.heads_major:
                caches.append(sentinel((self.HK, self.rows, self.D), self.kind).permute(1, 0, 2))
            else:
                caches.append(sentinel((self.rows, self.HK, self.D), self.kind))
        i32 = lambda v: t.tensor(v, dtype=t.int32, device="cuda")
        q, k, v = self.parts(self.row.cuda())
        return dict(q=q, k=k, v=v, offsets=i32(self.off), inv_freq=self.inv_freq.cuda(),
                    q_weight=None if self.w[0] is None else self.w[0].cuda(),
                    k_weight=None if self.w[1] is None else self.w[1].cuda(), past=i32(self.past),
                    positions=i32(self.first), kv_begin=t.tensor(self.begin, device="cuda"),
                    q_out=sentinel((self.N, self.H, self.D), self.kind), k_out=caches[0], v_out=caches[1])

    def call(self, x, **kw):
        import gated_delta_rule_varlen_amd as gdn

        x = {**x, **kw}
        args = [x.pop(n) for n in ("q", "k", "v", "offsets")]
        return gdn.qk_norm_rope_varlen(*args, **x)

    def ref(self, interleaved, eps=1e-6):
        t = self.torch
        pos = t.cat([f + t.arange(n, dtype=t.float64) for f, n in zip(self.first, self.T)])
        q, k, v = self.parts(self.row)
        kw = dict(eps=eps, interleaved=interleaved, kind=self.kind)
        return rope_ref(q, self.w[0], pos, self.inv_freq, **kw), rope_ref(k, self.w[1], pos, self.inv_freq, **kw), v

    def places(self):
        return self.torch.cat([b + p + self.torch.arange(n) for b, p, n in zip(self.begin, self.past, self.T)])

    def check(self, interleaved):
        t = self.torch
        print(f"[case] {self.kind} H {self.H} HK {self.HK} D {self.D} rot {self.rot} T {self.T[:10]}", flush=True)
        x = self.dev()
        before = [c.clone() for c in (x["k_out"], x["v_out"])]
        q, k, v = self.call(x, interleaved=interleaved)
        t.cuda.synchronize()
        (rq, tq), (rk, tk), rv = self.ref(interleaved)
        at = self.places().cuda()
        assert_within(q, rq, tq, "q")
        assert_within(k[at], rk, tk, "k")
        assert (bits(v[at]) == bits(rv)).all(), "v is copied"
        rest = t.ones(self.rows, dtype=t.bool, device="cuda")
        rest[at] = False
        for c, b in zip((k, v), before):
            assert (bits(c[rest]) == bits(b[rest])).all(), "other rows stay"


RAGGED = dict(T=[0, 3, 1, 0, 0, 70, 2, 0], past=[4, 0, 9, 0, 3, 5, 1, 0])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("H,HK,D,rot", [(4, 2, 128, 128), (4, 1, 64, 64), (2, 2, 256, 64), (3, 1, 96, 48), (5, 1, 72, 72),
                                        (2, 1, 80, 40), (2, 1, 192, 96), (1, 1, 32, 2), (2, 1, 64, 0), (2, 1, 64, 50),
                                        (1, 3, 8, 6), (3, 2, 256, 254), (2, 2, 128, 32)])
def test_widths_and_types(torch, kind, interleaved, H, HK, D, rot):
    Case(torch, kind, H, HK, D, rot, seed=D + rot, **RAGGED).check(interleaved)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("first", [[1 << 20, 12345678], [(1 << 31) - 100, 4_000_000]])
def test_far_positions(torch, kind, first):
    Case(torch, kind, 2, 1, 64, 64, [40, 9], [0, 3], first=first).check(False)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [[1], [1] * 64, [1200, 900], [1] * 700, [5, 0] * 300])
def test_batches(torch, kind, T):
    Case(torch, kind, 2, 1, 64, 32, T, [i % 5 for i in range(len(T))]).check(False)


@pytest.mark.parametrize("kind", KINDS)
def test_options(torch, kind):
    """No weights, heads-major caches, in place, without values, packed rows, positions = past."""
    c = Case(torch, kind, 4, 2, 64, 64, seed=3, weights=False, heads_major=True, **RAGGED)
    c.check(False)
    c = Case(torch, kind, 4, 2, 64, 64, seed=3, **RAGGED)
    x = c.dev()
    q, k, v = c.call(x)
    in_place, k2, v2 = c.call(x, q_out=x["q"], positions=None)
    assert in_place.data_ptr() == x["q"].data_ptr() and (bits(in_place) == bits(q)).all()
    assert (bits(k2) == bits(k)).all() and (bits(v2) == bits(v)).all()
    x = c.dev()
    packed_q, packed_k, packed_v = c.call(x, kv_begin=None, q_out=None, k_out=None, v_out=None)
    at = c.places().cuda()
    assert (bits(packed_q) == bits(q)).all() and (bits(packed_k) == bits(k[at])).all()
    assert (bits(packed_v) == bits(x["v"])).all()
    only_q, only_k, none = c.call(x, kv_begin=None, v=None, q_out=None, k_out=None, v_out=None)
    assert none is None and (bits(only_q) == bits(q)).all() and (bits(only_k) == bits(packed_k)).all()


@pytest.mark.parametrize("kind", KINDS)
def test_rows_of_zeros_and_large_values(torch, kind):
    c = Case(torch, kind, 2, 1, 64, 64, [4], [0])
    c.row[0] = 0
    c.row[1] *= 100
    c.check(False)


@pytest.mark.parametrize("what", ["ok", "start", "end", "falling", "past", "begin", "run", "far"])
def test_malformed_calls_write_nothing(torch, what):
    c = Case(torch, "bf16", 2, 1, 64, 64, [3, 2, 40], [1, 0, 2])
    x = c.dev()
    for name, at, value in dict(ok=[], start=[("offsets", 0, 1)], end=[("offsets", 3, c.N + 1)],
                                falling=[("offsets", 1, c.N + 5)], past=[("past", 0, -1)], begin=[("kv_begin", 1, -1)],
                                run=[("kv_begin", 2, c.rows - 41)], far=[("kv_begin", 0, (1 << 63) - 2)])[what]:
        x[name][at] = value
    outs = [x[n] for n in ("q_out", "k_out", "v_out")]
    want = [bits(t).copy() for t in outs]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.call(x, dev_status=st)
    torch.cuda.synchronize()
    assert st.item() == (0 if what == "ok" else -9)
    for t, w in zip(outs, want):
        assert (bits(t) == w).all() == (what != "ok")


def test_calls_without_tokens(torch):
    c = Case(torch, "bf16", 2, 1, 64, 64, [0, 0], [1, 0])
    st = torch.ones(1, dtype=torch.int32, device="cuda")
    q, k, v = c.call(c.dev(), dev_status=st)
    torch.cuda.synchronize()
    assert q.shape == (0, 2, 64) and st.item() == 0


def test_graph_replays(torch):
    c = Case(torch, "bf16", 4, 2, 128, 64, [1, 1, 1], [5, 0, 9])
    x = c.dev()
    graph = torch.cuda.CUDAGraph()
    c.call(x)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        c.call(x)
    for turn in range(3):
        x["positions"].add_(100)
        x["q"].mul_(1.5)
        want = c.call({**x, "q_out": torch.empty_like(x["q_out"])})[0]
        torch.cuda.synchronize()
        x["q_out"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert (bits(x["q_out"]) == bits(want)).all()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,rot", [(64, 50), (256, 254), (72, 72), (8, 6)])
@pytest.mark.parametrize("T", [[3, 0, 9], [700, 613]])
def test_in_place_where_halves_are_no_pieces(torch, kind, D, rot, T):
    """q_out = q where an element's partner lies in another lane's piece."""
    c = Case(torch, kind, 5, 2, D, rot, T, [i % 3 for i in range(len(T))], seed=rot)
    q, _, _ = c.call(c.dev())
    x = c.dev()
    in_place, _, _ = c.call(x, q_out=x["q"])
    assert in_place.data_ptr() == x["q"].data_ptr() and (bits(in_place) == bits(q)).all()

"""GPU tests of residual_norm and gated_norm against their formulas in 64 bits: types, widths from one piece of a row to the
largest, strides, optional arguments, aliases, extreme values, streams and graphs."""
import pytest

from attn_util import DT, assert_within
from fp4_util import gated_ref, residual_ref, strided
from gpu_util import bits, ensure_built, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    ensure_built()
    return require_gpu()


def normal(torch, seed, *shape, kind="f32", scale=1.0):
    return (scale * torch.randn(shape, generator=torch.Generator().manual_seed(seed))).to(DT[kind])


def residual_case(torch, kind, stream, N, C, post=True, channels=True, weighted=True, with_residual=True, scale=0.7, wide=False,
                  eps=1e-6):
    import gated_delta_rule_varlen_amd as gdn

    x = normal(torch, 1, N, C, kind=kind)
    r = normal(torch, 2, N, C, kind=stream, scale=3.0) if with_residual else None
    w, p = (1 + normal(torch, s, C, scale=0.2) for s in (3, 4))
    c = 0.5 + normal(torch, 5, C, scale=0.1)
    w, p, c = w if weighted else None, p if post else None, c if channels else None

    def dev(t):
        if t is None:
            return None
        if not wide or t.dim() == 1:
            return t.to("cuda")
        room = torch.full((N, C + 16), float("nan"), dtype=t.dtype, device="cuda")  # rows of a wider buffer
        room[:, 8:8 + C] = t
        return room[:, 8:8 + C]

    kw = dict(weight=dev(w), post_weight=dev(p), scale=scale, channel_scale=dev(c), eps=eps)
    ro = None if with_residual else torch.empty((N, C), dtype=DT[stream], device="cuda")
    out, nxt = gdn.residual_norm(dev(x), dev(r), residual_out=ro, **kw)
    assert out.dtype == DT[kind] and nxt.dtype == DT[stream]
    y, h, y_tol, h_tol = residual_ref(x, r, w, p, scale, c, eps, kind, stream)
    what = f"residual {kind} {stream} N={N} C={C}"
    assert_within(out, y, y_tol, what + " out")
    assert_within(nxt, h, h_tol, what + " stream")
    return dev(x), dev(r), kw, out, nxt


# widths on both sides of every change of threads and pieces a row
@pytest.mark.parametrize("C", [8, 64, 504, 512, 520, 2048, 2056, 4096, 4104, 8192, 8200, 16384, 32760, 32768])
@pytest.mark.parametrize("kind,stream", [("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f16", "f32"), ("f32", "f32")])
def test_residual_widths(torch, kind, stream, C):
    residual_case(torch, kind, stream, 3, C)


@pytest.mark.parametrize("C", [4, 252, 256, 260, 1020, 1028, 16388])
def test_residual_widths_of_single_precision(torch, C):
    residual_case(torch, "f32", "f32", 5, C)


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("channels", [False, True])
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("with_residual", [False, True])
def test_residual_options(torch, post, channels, weighted, with_residual):
    for kind, stream in (("bf16", "f32"), ("f16", "f16")):
        residual_case(torch, kind, stream, 7, 640, post, channels, weighted, with_residual, scale=-1.3, wide=True)


@pytest.mark.parametrize("N", [1, 2, 5, 1000, 5001])
def test_residual_rows(torch, N):
    residual_case(torch, "bf16", "bf16", N, 136, wide=True)
    residual_case(torch, "f16", "f32", N, 1032)


def test_residual_in_place_and_without_the_stream(torch):
    import gated_delta_rule_varlen_amd as gdn

    for kind, stream in (("bf16", "bf16"), ("f16", "f32"), ("f32", "f32")):
        x, r, kw, out, nxt = residual_case(torch, kind, stream, 33, 1064)
        x2, r2 = x.clone(), r.clone()
        a, b = gdn.residual_norm(x2, r2, out=x2, residual_out=r2, **kw)
        assert a is x2 and b is r2
        assert (bits(x2) == bits(out)).all() and (bits(r2) == bits(nxt)).all()
        a, b = gdn.residual_norm(x, r, write_residual=False, **kw)
        assert b is None and (bits(a) == bits(out)).all()


def test_residual_rows_of_zeros_and_of_no_numbers(torch):
    import gated_delta_rule_varlen_amd as gdn

    x = torch.zeros(6, 256, dtype=torch.bfloat16, device="cuda")
    x[2, 7], x[4, 100] = float("nan"), float("inf")
    out, nxt = gdn.residual_norm(x, torch.zeros_like(x), weight=torch.ones(256, device="cuda"))
    assert (out[[0, 1, 3, 5]] == 0).all() and (nxt[[0, 1, 3, 5]] == 0).all()
    assert torch.isnan(out[2]).all() and torch.isnan(out[4, 100]) and torch.isinf(nxt[4, 100])
    x[:] = 1.0  # a scale of zero leaves the stream alone
    r = torch.randn(6, 256, device="cuda")
    assert (gdn.residual_norm(x, r, scale=0.0)[1] == r).all()


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_residual_large_and_small_numbers(torch, kind):
    import gated_delta_rule_varlen_amd as gdn

    big = 1e4 if kind == "f16" else 1e16
    for size in (big, 1 / big):
        x = normal(torch, 9, 4, 512, kind=kind, scale=size)
        out, nxt = gdn.residual_norm(x.cuda(), None, post_weight=torch.ones(512, device="cuda"), eps=0.0)
        ref = residual_ref(x, None, None, torch.ones(512), 1.0, None, 0.0, kind, kind)
        assert_within(out, ref[0], ref[2], f"{kind} numbers of {size}")


def gated_case(torch, kind, N, H, V, activation="silu", gate_first=False, norm=True, weighted=True, layouts=("rows", "rows"), seed=1,
               gate_scale=2.0):
    import gated_delta_rule_varlen_amd as gdn

    x, g = normal(torch, seed, N, H, V, kind=kind), normal(torch, seed + 1, N, H, V, kind=kind, scale=gate_scale)
    w = 1 + normal(torch, seed + 2, V, scale=0.2) if weighted and norm else None
    kw = dict(weight=None if w is None else w.cuda(), activation=activation, gate_first=gate_first, norm=norm)
    xd, gd = strided(x, layouts[0]), strided(g, layouts[1])
    out = gdn.gated_norm(xd, gd, **kw)
    y, tol = gated_ref(x, g, w, 1e-6, activation, gate_first, norm, kind)
    assert_within(out, y, tol, f"gated {kind} N={N} H={H} V={V} {activation}")
    return xd, gd, kw, out


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("V", [8, 24, 32, 40, 64, 72, 128, 136, 256, 264, 512, 520, 1000, 1024, 1032, 2040, 2048])
def test_gated_widths(torch, kind, V):
    gated_case(torch, kind, 5, 3, V)


@pytest.mark.parametrize("V", [4, 12, 20, 68, 132, 260, 516, 1028])
def test_gated_widths_of_single_precision(torch, V):
    gated_case(torch, "f32", 5, 3, V)


@pytest.mark.parametrize("activation", ["silu", "sigmoid"])
@pytest.mark.parametrize("gate_first", [False, True])
@pytest.mark.parametrize("norm,weighted", [(True, True), (True, False), (False, False)])
def test_gated_options(torch, activation, gate_first, norm, weighted):
    for kind in ("bf16", "f32"):
        gated_case(torch, kind, 9, 4, 128, activation, gate_first, norm, weighted, layouts=("heads", "wide"))


@pytest.mark.parametrize("N,H", [(1, 1), (1, 7), (3, 1), (17, 5), (2000, 3), (700, 32)])
def test_gated_rows(torch, N, H):
    gated_case(torch, "bf16", N, H, 64, layouts=("wide", "heads"))
    gated_case(torch, "f16", N, H, 256, "sigmoid", True)


def test_gated_in_place(torch):
    import gated_delta_rule_varlen_amd as gdn

    x, g, kw, out = gated_case(torch, "bf16", 50, 6, 192)
    for which in range(2):
        a = [x.clone(), g.clone()]
        y = gdn.gated_norm(*a, out=a[which], **kw)
        assert y is a[which] and (bits(y) == bits(out)).all()


def test_gates_far_out(torch):
    """Gates past the exponential's range on both sides, and infinite ones."""
    import gated_delta_rule_varlen_amd as gdn

    gated_case(torch, "f32", 4, 2, 64, gate_scale=100.0)
    x = torch.ones(1, 1, 8, device="cuda")
    g = torch.tensor([200.0, -200.0, float("inf"), -float("inf"), 0.0, 1e30, -1e30, 88.0], device="cuda").view(1, 1, 8)
    y = gdn.gated_norm(x, g, activation="sigmoid", norm=False).flatten().tolist()
    assert y[:7] == [1.0, 0.0, 1.0, 0.0, 0.5, 1.0, 0.0]
    y = gdn.gated_norm(x, g, norm=False).flatten().tolist()
    assert y[0] == 200.0 and y[1] == 0.0 and y[2] == float("inf") and y[4] == 0.0 and y[6] == 0.0


def test_norms_on_another_stream_and_in_a_graph(torch):
    import gated_delta_rule_varlen_amd as gdn

    x, r, kw, out, nxt = residual_case(torch, "bf16", "f32", 300, 2048)
    gx, gg, gkw, gout = gated_case(torch, "bf16", 300, 16, 128)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o1, o2, o3 = torch.empty_like(out), torch.empty_like(nxt), torch.empty_like(gout)
    with torch.cuda.stream(side):
        gdn.residual_norm(x, r, out=o1, residual_out=o2, **kw)
        gdn.gated_norm(gx, gg, out=o3, **gkw)
    side.synchronize()
    same = lambda: (bits(o1) == bits(out)).all() and (bits(o2) == bits(nxt)).all() and (bits(o3) == bits(gout)).all()
    assert same()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gdn.residual_norm(x, r, out=o1, residual_out=o2, **kw)
        gdn.gated_norm(gx, gg, out=o3, **gkw)
    for _ in range(3):
        for o in (o1, o2, o3):
            o.fill_(7.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert same()

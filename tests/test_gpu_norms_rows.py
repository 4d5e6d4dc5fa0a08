"""GPU tests of residual_norm where a block goes over several rows, at every width's threads and pieces a row: the sums of one
row after the other share their places in LDS, and a row is fetched while another is worked on."""
import pytest

from attn_util import DT, assert_within
from fp4_util import residual_ref
from gpu_util import bits, ensure_built, require_gpu
from test_gpu_norms import normal

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    ensure_built()
    return require_gpu()


# (type, stream, width, rows): three rows a block or more, of 1024 blocks of 256 threads, 512 of 512 and 256 of 1024
LOOPS = [("bf16", "bf16", 512, 12301), ("bf16", "f32", 2048, 3077), ("f16", "f16", 4096, 3077), ("bf16", "f32", 8192, 1541),
         ("f16", "f32", 16384, 777), ("bf16", "bf16", 32768, 777), ("bf16", "f32", 32768, 777), ("f32", "f32", 4096, 1541),
         ("f32", "f32", 16384, 777), ("f32", "f32", 32768, 777)]


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("kind,stream,C,N", LOOPS)
def test_blocks_of_several_rows(torch, kind, stream, C, N, post):
    """Rows of sizes that differ by up to 2^6, so that a sum of another row shows.  The whole output against the
    operator on single rows (a block each), those against the formula, and the call in place."""
    import gated_delta_rule_varlen_amd as gdn

    size = torch.exp2(torch.arange(N) % 7.0)[:, None]
    x = (normal(torch, 11, N, C) * size).to(DT[kind])
    r = (normal(torch, 12, N, C) * size).to(DT[stream])
    w, p = (1 + normal(torch, s, C, scale=0.2) for s in (13, 14))
    kw = dict(weight=w.cuda(), post_weight=p.cuda() if post else None, scale=0.7)
    xd, rd = x.cuda(), r.cuda()
    out, nxt = gdn.residual_norm(xd, rd, **kw)
    for first in range(0, N, 200):  # 200 rows of any width are a block each, or a wave each
        a, b = gdn.residual_norm(xd[first:first + 200], rd[first:first + 200], **kw)
        assert (bits(out[first:first + 200]) == bits(a)).all() and (bits(nxt[first:first + 200]) == bits(b)).all(), f"rows from {first}"
    some = torch.arange(0, N, max(1, N // 40))
    y, h, y_tol, h_tol = residual_ref(x[some], r[some], w, p if post else None, 0.7, None, 1e-6, kind, stream)
    assert_within(out[some.cuda()], y, y_tol, f"{kind} {stream} {C} out")
    assert_within(nxt[some.cuda()], h, h_tol, f"{kind} {stream} {C} stream")
    gdn.residual_norm(xd, rd, out=xd, residual_out=rd, **kw)
    assert (bits(xd) == bits(out)).all() and (bits(rd) == bits(nxt)).all()


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("with_residual", [False, True])
def test_both_outputs_of_large_and_small_numbers(torch, kind, with_residual):
    import gated_delta_rule_varlen_amd as gdn

    big = 1e4 if kind == "f16" else 1e16
    for size in (big, 1 / big):
        x = normal(torch, 9, 4, 512, kind=kind, scale=size)
        r = normal(torch, 10, 4, 512, kind=kind, scale=size) if with_residual else None
        out, nxt = gdn.residual_norm(x.cuda(), None if r is None else r.cuda(), weight=torch.ones(512, device="cuda"), scale=0.5, eps=0.0)
        ref = residual_ref(x, r, torch.ones(512), None, 0.5, None, 0.0, kind, kind)
        assert_within(out, ref[0], ref[2], f"{kind} numbers of {size}")
        assert_within(nxt, ref[1], ref[3], f"{kind} stream of numbers of {size}")

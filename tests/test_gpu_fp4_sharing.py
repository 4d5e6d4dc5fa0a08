"""GPU tests of attention_fp4_varlen where sequences share rows of the cache, and where queries hold no numbers."""
import pytest

from attn_util import assert_within, attention_ref
from gpu_util import ensure_built, require_gpu
from test_gpu_fp4_attention import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    ensure_built()
    return require_gpu()


# types, key heads, query heads of each, head width, new tokens, keys, sequences that share them
SHARED = [("bf16", 2, 4, 64, 1, 300, 9), ("f16", 2, 4, 128, 1, 2900, 40), ("bf16", 2, 8, 256, 5, 1000, 30), ("f32", 1, 8, 160, 9, 700, 12),
          ("f32", 2, 2, 64, 3, 500, 300), ("bf16", 2, 2, 128, 70, 500, 7), ("f32", 1, 2, 256, 60, 200, 5)]


@pytest.mark.parametrize("kind,HK,G,D,T,n,B", SHARED)
def test_sequences_over_the_same_rows(torch, kind, HK, G, D, T, n, B):
    """Every sequence reads the one run, or a part of it that begins inside: more tiles than the cache has rows for."""
    c = Case(torch, kind, HK, G, D, [(T, n)] + [(T, 0)] * (B - 1))
    c.begin = [c.begin[0] + (b % 3) * 17 for b in range(B)]
    c.n = [n - (b % 3) * 17 - b % 5 for b in range(B)]
    c.check(f"{B} sequences over {n} rows, {kind} {D}")


@pytest.mark.parametrize("kind", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("D,G,lengths", [(64, 4, [(4, 40), (1, 300)]), (128, 8, [(5, 3000), (2, 40)]), (256, 8, [(5, 4000), (2, 40)]),
                                         (128, 4, [(90, 300)]), (256, 4, [(90, 300), (40, 70)])])
def test_queries_without_numbers(torch, kind, bad, D, G, lengths):
    """A query that is no number, or infinite, spoils its own row and no other."""
    import gated_delta_rule_varlen_amd as gdn

    c = Case(torch, kind, 2, G, D, lengths)
    want, stats = c.check("clean")
    row, head = 1, G + 1
    c.q[row, head, 5] = bad
    out, lse = gdn.attention_fp4_varlen(**c.dev(), max_q=max(c.T), return_lse=True)
    hit = torch.zeros(out.shape[:2], dtype=torch.bool, device="cuda")
    hit[row, head] = True
    assert torch.isnan(out[hit]).all() and not torch.isfinite(lse[hit]).any()
    # the others within the bounds of the plain form: a row's neighbours may decide when its sums are scaled
    k, v = c.values()
    q = c.q.clone()
    q[row, head] = 0.0
    ref = attention_ref(q, k, v, c.T, c.begin, c.n, kind=c.kind)
    by, rest = 3.0 if kind == "f32" else 1.0, ~hit.cpu()
    assert_within(out.cpu()[rest], ref[0][rest], by * ref[2][rest], f"{kind} {D} out")
    assert_within(lse.cpu()[rest], ref[1][rest], by * ref[3][rest], f"{kind} {D} lse")

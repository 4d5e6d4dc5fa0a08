"""GPU tests of attention_fp4_varlen where a cache's scales leave the range of the operands.  With fp16 queries values are
operands in fp16, so those of scale bytes from 141 on may be infinite (6 * 2^14 is); with the others, whose operands have
fp32's range, those of 253 and 254."""
import pytest

from attn_util import DT, assert_within, attention_ref
from fp4_util import decode
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

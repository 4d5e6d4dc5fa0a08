"""GPU tests of the attention's larger forms against the plain 64-bit attention: more sequences than a wave has lanes
and than one read of the call's arrays holds, prefixes whose launches are split, tiles of eight waves, and
sequences that go by their length."""
import pytest

from gpu_util import bits, ensure_built, require_gpu
from test_gpu_attention import KINDS, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    ensure_built()
    return require_gpu()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B", [63, 64, 65, 256, 257, 700])
def test_single_tokens_of_many_sequences(torch, kind, B):
    Case(torch, kind, 1, 2, 64, [(i % 3 != 1, 1 + (37 * i) % 90) for i in range(B)], seed=B).check(f"{B} sequences")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B", [2, 64, 65, 130])
@pytest.mark.parametrize("D", [64, 256])
def test_prompts_of_many_sequences(torch, kind, B, D):
    """Rows of more than one tile: up to 64 sequences go by their keys, equal ones among them."""
    Case(torch, kind, 2, 4, D, [(0 if i % 7 == 3 else 20 + (i * 29) % 60, 90 + 10 * (i % 5)) for i in range(B)],
         seed=B).check(f"{B} prompts D{D}")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("HK,G,D,T", [(4, 2, 64, 1), (4, 4, 128, 1), (2, 8, 128, 5), (2, 2, 256, 1), (1, 16, 64, 4)])
def test_prefix_of_many_sequences(torch, kind, HK, G, D, T):
    """More blocks than run at once, so prefix and own keys take a launch each."""
    Case(torch, kind, HK, G, D, [(T, T + (53 * i) % 200) for i in range(150)], prefix=333, seed=D).check(f"prefix of many D{D}")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("HK,G,lengths", [(2, 1, [(700, 700), (129, 400)]), (1, 8, [(260, 1300)]), (1, 5, [(103, 103), (52, 60)])])
@pytest.mark.parametrize("D", [128, 200, 256])
def test_wide_heads_over_several_tiles(torch, kind, HK, G, lengths, D):
    Case(torch, kind, HK, G, D, lengths, seed=D).check(f"wide D{D}")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_masked_values_of_long_prompts(torch, kind, value, D):
    """Values that are not finite in the last rows of a long prompt, over several row tiles of every width."""
    c = Case(torch, kind, 1, 4, D, [(150, 300), (90, 90)], seed=8)
    for b, (_, n) in enumerate(c.lengths):
        for x in c.kv:
            x[c.begin[b] + n - 1] = value
    out, lse = c.call()
    o, l, ot, lt = c.ref()
    keep = torch.ones(c.N, dtype=torch.bool)
    keep[[149, 239]] = False
    from attn_util import assert_within

    assert_within(out[keep.cuda()], o[keep], ot[keep], "masked out")
    assert_within(lse[keep.cuda()], l[keep], lt[keep], "masked lse")


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_joint_and_separate_launches_repeat(torch, kind):
    for B in (6, 150):
        c = Case(torch, kind, 2, 4, 128, [(2, 60 + i % 50) for i in range(B)], prefix=700, seed=B)
        x = c.dev()
        first, second = c.call(x), c.call(x)
        torch.cuda.synchronize()
        for a, b in zip(first, second):
            assert (bits(a) == bits(b)).all()

"""GPU tests of gdn_qk_norm_rope_varlen where keys and values share or straddle the passes of a wave (16 rows of
64 half-precision elements, fewer of wider ones), with and without values, few tokens and many."""
import pytest

from attn_util import assert_within
from gpu_util import bits, ensure_built, require_gpu
from test_gpu_rope import KINDS, Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    ensure_built()
    return require_gpu()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("H,HK", [(17, 1), (6, 3), (16, 8), (9, 9), (33, 11), (1, 20)])
@pytest.mark.parametrize("D,rot", [(64, 64), (128, 32), (256, 256)])
def test_keys_and_values_of_a_pass(torch, kind, interleaved, H, HK, D, rot):
    Case(torch, kind, H, HK, D, rot, [3, 0, 1, 20], [0, 7, 2, 1], seed=H + HK).check(interleaved)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("HK", [1, 3, 9])
def test_many_tokens(torch, kind, HK):
    Case(torch, kind, 2, HK, 64, 32, [700, 0, 813], [4, 1, 0], seed=HK).check(False)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("HK,D", [(3, 64), (9, 64), (5, 128)])
def test_without_values(torch, kind, HK, D):
    c = Case(torch, kind, 4, HK, D, 32, [5, 30], [0, 3], seed=HK)
    x = c.dev()
    before = x["v_out"].clone()
    q, k, none = c.call(x, v=None, v_out=None)
    (rq, tq), (rk, tk), _ = c.ref(False)
    assert none is None and (bits(x["v_out"]) == bits(before)).all()
    assert_within(q, rq, tq, "q")
    assert_within(k[c.places().cuda()], rk, tk, "k")

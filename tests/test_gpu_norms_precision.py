"""GPU tests of gated_norm in fp32: gates of every size to a few roundings."""
import pytest

from attn_util import E32, assert_within
from fp4_util import strided
from gpu_util import ensure_built, require_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    ensure_built()
    return require_gpu()


@pytest.mark.parametrize("activation", ["silu", "sigmoid"])
def test_single_precision_gates_of_every_size(torch, activation):
    """act(g) itself (x = 1, no norm), also where exp(-g) passes fp32.  The exponential is off by 3 units of its last place
    (6 e), the sum, the quotient and the product with g by e each, the product with x by none; numbers below the normal
    range by half of the smallest one in the exponential, twice (it is a summand of at most 1 and the result), times |g|, and
    in the product."""
    import gated_delta_rule_varlen_amd as gdn

    g = torch.cat([torch.linspace(-110, 110, 40001), torch.linspace(-4, 4, 9999), torch.tensor([0.0, -0.0, 1e-30, -1e-30, 1e30, 60000.0])])
    g = torch.nn.functional.pad(g, (0, -len(g) % 128)).view(-1, 1, 128)
    out = gdn.gated_norm(torch.ones_like(g).cuda(), g.cuda(), activation=activation, norm=False)
    ref = torch.sigmoid(g.double())
    size = torch.ones_like(ref)
    if activation == "silu":
        ref, size = ref * g.double(), g.double().abs().clamp(min=1.0)
    assert_within(out, ref, 9 * E32 * ref.abs() + 2.0 ** -148 * size, f"{activation} in fp32")


def test_single_precision_gates_beside_the_norm(torch):
    """Gates far on the negative side, where an argument that is rounded before the exponential shows."""
    import gated_delta_rule_varlen_amd as gdn

    gen = torch.Generator().manual_seed(3)
    x, g = torch.randn(7, 3, 64, generator=gen), -80 + 3 * torch.randn(7, 3, 64, generator=gen)
    out = gdn.gated_norm(strided(x, "heads"), strided(g, "wide"), eps=0.0)
    y = x.double()
    y = y / torch.sqrt(y.square().mean(-1, keepdim=True)) * g.double() * torch.sigmoid(g.double())
    # the gate by 9 e, the norm by 43 + 8 e (half of its sum's 86, its root, the quotient and the products), their product by 1
    assert_within(out, y, 60 * 1.01 * E32 * y.abs() + 2.0 ** -148, "gates far down")

"""GPU tests of the 4-bit cache whose rows lie as far apart as a call may say: the offsets inside a tile's range stay in bounds and
reach their rows in every form, and bytes between the rows are left alone."""
import pytest

from attn_util import assert_within, attention_ref
from fp4_util import decode
from gpu_util import ensure_built, require_gpu
from test_gpu_fp4_attention import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    ensure_built()
    return require_gpu()


@pytest.mark.parametrize("kind,G,D,lengths", [
    ("bf16", 4, 64, [(1, 700), (1, 30)]),      # a block a run
    ("bf16", 4, 128, [(1, 2500), (1, 33)]),    # cut and joined
    ("f32", 8, 64, [(5, 1500)]),               # several row tiles
    ("bf16", 8, 256, [(6, 900)]),              # two groups of waves
    ("bf16", 2, 128, [(100, 900), (3, 40)]),   # prompts
    ("f32", 2, 64, [(100, 900)]),
])
@pytest.mark.parametrize("scales_apart", [2**20, 2**20 - 1])
def test_rows_a_mebibyte_apart(torch, kind, G, D, lengths, scales_apart):
    import gated_delta_rule_varlen_amd as gdn

    c = Case(torch, kind, 1, G, D, lengths)
    rows = len(c.cache[0])
    x = c.dev()
    far = []
    for i, part in enumerate(c.cache):
        apart = 2**20 if i % 2 == 0 else scales_apart
        room = torch.full((rows * apart + 4096,), 255, dtype=torch.uint8, device="cuda")
        view = room.as_strided((rows, 1, part.shape[2]), (apart, part.shape[2], 1))
        view.copy_(part)
        far.append(view)
    x["cache"] = tuple(far)
    out, lse = gdn.attention_fp4_varlen(**x, max_q=max(c.T), return_lse=True)
    k, v = c.values()
    ref = attention_ref(c.q, k, v, c.T, c.begin, c.n, kind=kind)
    by = 3.0 if kind == "f32" else 1.0
    assert_within(out, ref[0], by * ref[2], f"far rows {kind} {D} out")
    assert_within(lse, ref[1], by * ref[3], f"far rows {kind} {D} lse")
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    rk, rv = gdn.cache_read_fp4_varlen(x["cache"], off, N=rows, dtype=torch.float32)
    used = ~torch.isnan(k)
    assert torch.equal(rk.cpu().double()[used], decode(*c.cache[:2])[used])
    assert torch.equal(rv.cpu().double()[used], v[used])
    del far, x
    torch.cuda.empty_cache()

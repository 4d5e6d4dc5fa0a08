"""The 4-bit cache and the block's norms on the host: the references pin the format, and every bad argument gets its status
before anything is launched (device pointers are stand-in addresses that are never dereferenced)."""
import ctypes

import pytest
import torch

from fp4_util import decode, encode
from gpu_util import ensure_built

P = 0x10000


@pytest.fixture(scope="module")
def abi():
    ensure_built()
    from gated_delta_rule_varlen_amd import _abi

    _abi.lib()
    return _abi


# ---- the references --------------------------------------------------------------------------------
def block(*values):
    x = torch.zeros(32, dtype=torch.float64)
    x[: len(values)] = torch.tensor(values, dtype=torch.float64)
    return x


def test_values_of_the_codes_come_back():
    x = block(0.5, -0.5, 1, 1.5, -2, 3, 4, 6, -6)
    for e in (-100, -3, 0, 7, 100):
        codes, scales = encode(x * 2.0**e, "f32")
        assert scales.item() == 127 + e
        assert torch.equal(decode(codes, scales), x * 2.0**e)


def test_first_element_is_the_low_half():
    codes, scales = encode(block(6, -1), "f32")
    assert codes[0].item() == 7 | (10 << 4) and codes[1:].sum() == 0 and scales.item() == 127


@pytest.mark.parametrize("x,want", [(0.25, 0), (0.75, 1), (1.25, 1), (1.75, 2), (2.5, 2), (3.5, 4), (5, 4), (0.26, 0.5),
                                    (0.74, 0.5), (-2.51, -3), (4.99, 4), (5.01, 6)])
def test_ties_go_to_the_even_code(x, want):
    codes, scales = encode(block(6, x), "f32")
    assert decode(codes, scales)[1].item() == want


@pytest.mark.parametrize("top,e", [(6, 0), (6.0000001, 1), (3, -1), (3.0000001, 0), (12, 1), (2.0**-130, -126), (0, -126)])
def test_power_is_the_least_that_holds_the_block(top, e):
    assert encode(block(-top), "f32")[1].item() == 127 + e


def test_fp16_scales_keep_to_fp16_numbers():
    codes, scales = encode(block(65504.0, -1.0), "f16")
    assert scales.item() == 127 + 13 and decode(codes, scales)[0].item() == 49152
    codes, scales = encode(block(2.0**-24), "f16")
    assert scales.item() == 127 - 23 and decode(codes, scales)[0].item() == 2.0**-24  # half of 2^-23


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_block_without_numbers(bad):
    x = torch.cat((block(1, bad), block(1)))
    codes, scales = encode(x, "f32")
    assert scales.tolist() == [255, 125] and codes[:16].sum() == 0
    y = decode(codes, scales)
    assert torch.isnan(y[:32]).all() and y[32].item() == 1


# ---- refusals of the C ABI -------------------------------------------------------------------------
def make(cls, base, f):
    base.update(f)
    return cls(*[base[n] for n, _ in cls._fields_])


def cache_of(abi, **f):
    D = 64
    return make(abi.Fp4Cache, dict(k_codes=P, k_scales=P, v_codes=P, v_scales=P, rows=100, k_codes_stride=(D, D // 2),
                                   k_scales_stride=(D // 16, D // 32), v_codes_stride=(D, D // 2),
                                   v_scales_stride=(D // 16, D // 32)), f)


def rows_call(abi, read, fields, cache, k=P, v=P, off=P, past=None, begin=P):
    d = make(abi.Fp4RowsDesc, dict(B=2, N=8, HK=2, D=64, dtype=1, flags=0, k_stride=(128, 64), v_stride=(128, 64)), fields)
    L, d, c = abi.lib(), ctypes.byref(d), None if cache is None else ctypes.byref(cache)
    if read:
        return L.gdn_cache_read_fp4_varlen(d, c, off, past, begin, k, v, None, None)
    return L.gdn_cache_write_fp4_varlen(d, k, v, off, past, begin, c, None, None)


CACHE_REFUSALS = [
    (dict(rows=-1), "ERR_SHAPE"),
    (dict(rows=2**62), "ERR_OVERFLOW"),
    (dict(k_codes=None), "ERR_NULL"),
    (dict(k_scales=None), "ERR_NULL"),
    (dict(v_codes=None), "ERR_NULL"),
    (dict(v_scales=None), "ERR_NULL"),
    (dict(k_codes=P + 8), "ERR_ALIGN"),
    (dict(v_codes_stride=(72, 32)), "ERR_ALIGN"),
    (dict(k_codes_stride=(64, 40)), "ERR_ALIGN"),
    (dict(k_codes_stride=(-64, 32)), "ERR_SHAPE"),
    (dict(v_scales_stride=(4, -2)), "ERR_SHAPE"),
    (dict(v_codes_stride=(2**23, 32)), "ERR_OVERFLOW"),  # rows 8 MiB apart
    (dict(k_scales_stride=(2**23, 2)), "ERR_OVERFLOW"),
    (dict(v_codes_stride=(2**20 + 16, 32)), "ERR_OVERFLOW"),
    (dict(v_scales_stride=(2**20 + 1, 2)), "ERR_OVERFLOW"),
    (dict(k_codes_stride=(64, 2**61)), "ERR_OVERFLOW"),
]


@pytest.mark.parametrize("read", [False, True])
@pytest.mark.parametrize("fields,want", CACHE_REFUSALS)
def test_rows_refuse_a_cache(abi, read, fields, want):
    assert rows_call(abi, read, {}, cache_of(abi, **fields)) == getattr(abi, want)


@pytest.mark.parametrize("read", [False, True])
@pytest.mark.parametrize(
    "fields,kw,want",
    [
        (dict(B=0), {}, "ERR_SHAPE"),
        (dict(N=-1), {}, "ERR_SHAPE"),
        (dict(HK=0), {}, "ERR_SHAPE"),
        (dict(D=0), {}, "ERR_SHAPE"),
        (dict(D=48), {}, "ERR_SHAPE"),
        (dict(D=288), {}, "ERR_SHAPE"),
        (dict(N=2**31 - 100, HK=1), {}, "ERR_OVERFLOW"),
        (dict(N=2**30, HK=2), {}, "ERR_OVERFLOW"),
        (dict(N=2**27 - 7, HK=1), {}, "ERR_OVERFLOW"),
        (dict(dtype=3), {}, "ERR_DTYPE"),
        (dict(flags=1), {}, "ERR_UNSUPPORTED"),
        (dict(k_stride=(-128, 64)), {}, "ERR_SHAPE"),
        (dict(v_stride=(132, 64)), {}, "ERR_ALIGN"),
        (dict(N=101), dict(begin=None), "ERR_SHAPE"),  # row t of 100 rows
        ({}, dict(k=None), "ERR_NULL"),
        ({}, dict(v=None), "ERR_NULL"),
        ({}, dict(off=None), "ERR_NULL"),
        ({}, dict(k=P + 2), "ERR_ALIGN"),
    ],
)
def test_rows_refusals(abi, read, fields, kw, want):
    assert rows_call(abi, read, fields, cache_of(abi), **kw) == getattr(abi, want)
    assert rows_call(abi, read, {}, None) == abi.ERR_NULL


def attn_desc(abi, **f):
    none = (0, 0)
    return make(abi.AttnDesc, dict(B=2, N=8, H=8, HK=2, D=64, max_q=6, dtype=1, flags=0, scale=0.0, prefix_len=0, kv_rows=100,
                                   q_stride=(512, 64), k_stride=none, v_stride=none, out_stride=(512, 64), prefix_k_stride=none,
                                   prefix_v_stride=none), f)


def attention(abi, fields, cache, q=P, off=P, begin=P, length=P, out=P, ws=P, ws_bytes=1 << 40):
    return abi.lib().gdn_attention_fp4_varlen(ctypes.byref(attn_desc(abi, **fields)), q, None if cache is None else ctypes.byref(cache),
                                              off, begin, length, out, None, ws, ws_bytes, None, None)


@pytest.mark.parametrize("fields,want", CACHE_REFUSALS)
def test_attention_refuses_a_cache(abi, fields, want):
    rows = dict(kv_rows=fields["rows"]) if "rows" in fields else {}
    assert attention(abi, rows, cache_of(abi, **fields)) == getattr(abi, want)


@pytest.mark.parametrize(
    "fields,kw,want",
    [
        (dict(B=0), {}, "ERR_SHAPE"),
        (dict(N=-1), {}, "ERR_SHAPE"),
        (dict(HK=3), {}, "ERR_SHAPE"),
        (dict(D=48), {}, "ERR_SHAPE"),
        (dict(D=288), {}, "ERR_SHAPE"),
        (dict(max_q=0), {}, "ERR_SHAPE"),
        (dict(prefix_len=5), {}, "ERR_SHAPE"),
        (dict(kv_rows=99), {}, "ERR_SHAPE"),  # not the cache's
        (dict(scale=float("nan")), {}, "ERR_SHAPE"),
        (dict(dtype=3), {}, "ERR_DTYPE"),
        (dict(flags=1), {}, "ERR_UNSUPPORTED"),
        (dict(N=2**30), {}, "ERR_OVERFLOW"),
        (dict(q_stride=(-512, 64)), {}, "ERR_SHAPE"),
        (dict(out_stride=(512, 68)), {}, "ERR_ALIGN"),
        ({}, dict(q=None), "ERR_NULL"),
        ({}, dict(out=None), "ERR_NULL"),
        ({}, dict(off=None), "ERR_NULL"),
        ({}, dict(begin=None), "ERR_NULL"),
        ({}, dict(length=None), "ERR_NULL"),
        ({}, dict(q=P + 8), "ERR_ALIGN"),
        ({}, dict(ws=P + 4), "ERR_ALIGN"),
    ],
)
def test_attention_refusals(abi, fields, kw, want):
    assert attention(abi, fields, cache_of(abi), **kw) == getattr(abi, want)
    assert attention(abi, {}, None) == abi.ERR_NULL


@pytest.mark.parametrize("fields", [{}, dict(max_q=200, N=400, q_stride=(512, 64)), dict(dtype=0), dict(N=1, max_q=1, kv_rows=1 << 20)])
def test_attention_workspace(abi, fields):
    n = ctypes.c_size_t(77)
    d = attn_desc(abi, **fields)
    assert abi.lib().gdn_attention_fp4_workspace_bytes(ctypes.byref(d), ctypes.byref(n)) == abi.OK
    if n.value:  # too little of it is refused
        rows = fields.get("kv_rows", 100)
        for kw in (dict(ws=None), dict(ws_bytes=n.value - 1)):
            assert attention(abi, fields, cache_of(abi, rows=rows), **kw) == abi.ERR_WORKSPACE
    assert abi.lib().gdn_attention_fp4_workspace_bytes(ctypes.byref(d), None) == abi.ERR_NULL
    assert abi.lib().gdn_attention_fp4_workspace_bytes(None, ctypes.byref(n)) == abi.ERR_NULL


def residual(abi, fields, x=P, r=P, post=None, ch=None, w=P, out=P, ro=P):
    d = make(abi.ResidualNormDesc, dict(N=4, C=64, dtype=1, residual_dtype=1, eps=1e-6, scale=1.0, x_stride=64, residual_stride=64,
                                        out_stride=64, residual_out_stride=64), fields)
    return abi.lib().gdn_residual_norm(ctypes.byref(d), x, r, post, ch, w, out, ro, None)


@pytest.mark.parametrize(
    "fields,kw,want",
    [
        (dict(N=-1), {}, "ERR_SHAPE"),
        (dict(C=0), {}, "ERR_SHAPE"),
        (dict(C=32776), {}, "ERR_SHAPE"),
        (dict(eps=-1.0), {}, "ERR_SHAPE"),
        (dict(eps=float("nan")), {}, "ERR_SHAPE"),
        (dict(scale=float("inf")), {}, "ERR_SHAPE"),
        (dict(x_stride=56), {}, "ERR_SHAPE"),
        (dict(residual_out_stride=-64), {}, "ERR_SHAPE"),
        (dict(dtype=4), {}, "ERR_DTYPE"),
        (dict(residual_dtype=2), {}, "ERR_DTYPE"),
        (dict(dtype=0, residual_dtype=1), {}, "ERR_DTYPE"),
        (dict(N=2**31 - 1, x_stride=2**60), {}, "ERR_OVERFLOW"),
        (dict(C=60), {}, "ERR_ALIGN"),
        (dict(out_stride=68), {}, "ERR_ALIGN"),
        (dict(residual_dtype=0, residual_stride=66), {}, "ERR_ALIGN"),
        ({}, dict(x=None), "ERR_NULL"),
        ({}, dict(out=None), "ERR_NULL"),
        ({}, dict(x=P + 8), "ERR_ALIGN"),
        ({}, dict(w=P + 4), "ERR_ALIGN"),
        ({}, dict(post=P + 4), "ERR_ALIGN"),
        ({}, dict(ch=P + 4), "ERR_ALIGN"),
    ],
)
def test_residual_norm_refusals(abi, fields, kw, want):
    assert residual(abi, fields, **kw) == getattr(abi, want)


def test_no_tokens_launch_nothing(abi):
    assert residual(abi, dict(N=0), x=None, r=None, out=None, ro=None) == abi.OK
    assert gated(abi, dict(N=0), x=None, z=None, out=None) == abi.OK


def gated(abi, fields, x=P, z=P, w=P, out=P):
    d = make(abi.GatedNormDesc, dict(N=4, H=2, V=64, dtype=1, flags=0, eps=1e-6, x_stride=(128, 64), gate_stride=(128, 64),
                                     out_stride=(128, 64)), fields)
    return abi.lib().gdn_gated_norm(ctypes.byref(d), x, z, w, out, None)


@pytest.mark.parametrize(
    "fields,kw,want",
    [
        (dict(N=-1), {}, "ERR_SHAPE"),
        (dict(H=0), {}, "ERR_SHAPE"),
        (dict(V=0), {}, "ERR_SHAPE"),
        (dict(V=2056), {}, "ERR_SHAPE"),
        (dict(eps=-1.0), {}, "ERR_SHAPE"),
        (dict(x_stride=(-128, 64)), {}, "ERR_SHAPE"),
        (dict(dtype=3), {}, "ERR_DTYPE"),
        (dict(flags=8), {}, "ERR_UNSUPPORTED"),
        (dict(flags=4), {}, "ERR_UNSUPPORTED"),  # a weight without a norm
        (dict(N=2**30, H=2), {}, "ERR_OVERFLOW"),
        (dict(V=60), {}, "ERR_ALIGN"),
        (dict(gate_stride=(132, 64)), {}, "ERR_ALIGN"),
        ({}, dict(x=None), "ERR_NULL"),
        ({}, dict(z=None), "ERR_NULL"),
        ({}, dict(out=None), "ERR_NULL"),
        ({}, dict(z=P + 2), "ERR_ALIGN"),
        ({}, dict(w=P + 4), "ERR_ALIGN"),
    ],
)
def test_gated_norm_refusals(abi, fields, kw, want):
    assert gated(abi, fields, **kw) == getattr(abi, want)


# ---- what the binding turns away -------------------------------------------------------------------
def test_the_binding_takes_device_tensors_only(abi):
    import gated_delta_rule_varlen_amd as gdn

    off, x, y = torch.tensor([0, 4], dtype=torch.int32), torch.zeros(4, 2, 64), torch.zeros(4, 64)
    cache = [torch.zeros(9, 2, w, dtype=torch.uint8) for w in (32, 2, 32, 2)]
    at = dict(kv_len=off[1:], kv_begin=torch.zeros(1, dtype=torch.int64))
    for bad in (x, None, 3):
        with pytest.raises((TypeError, ValueError)):
            gdn.cache_write_fp4_varlen(bad, bad, off, cache=cache)
        with pytest.raises((TypeError, ValueError)):
            gdn.cache_read_fp4_varlen(cache, off, k_out=x if bad is None else bad)
        with pytest.raises((TypeError, ValueError)):
            gdn.attention_fp4_varlen(bad, cache, off, **at)
        with pytest.raises((TypeError, ValueError)):
            gdn.residual_norm(y if bad is x else bad)
        with pytest.raises((TypeError, ValueError)):
            gdn.gated_norm(bad, x)
    with pytest.raises(ValueError):
        gdn.gated_norm(x, x, activation="tanh")
    with pytest.raises(ValueError):
        gdn.cache_read_fp4_varlen(cache, off)  # how many tokens
    for bad in ((), cache[:3], tuple(cache) + (x,), [3] * 4, iter(cache), None, "abcd"):
        with pytest.raises((TypeError, ValueError)):
            gdn.cache_read_fp4_varlen(bad, off, N=4)
    with pytest.raises((TypeError, ValueError)):
        gdn.cache_read_fp4_varlen(cache, off, N=4, dtype=3)
    for rows, HK, D in ((-1, 1, 64), (5, 0, 64), (5, 1, 48), (5, 1, 288)):
        with pytest.raises(ValueError):
            gdn.fp4_cache(rows, HK, D, device="cpu")


def test_a_new_cache_lies_head_by_head(abi):
    import gated_delta_rule_varlen_amd as gdn

    c = gdn.fp4_cache(10, 3, 96, device="cpu")
    assert [tuple(x.shape) for x in c] == [(10, 3, 48), (10, 3, 3)] * 2
    assert [x.stride() for x in c] == [(48, 480, 1), (3, 30, 1)] * 2 and all(int(x.sum()) == 0 for x in c)

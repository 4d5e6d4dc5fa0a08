"""Refusals of the softmax-attention entry points, on the host: bad arguments get the documented status
before anything is launched (device pointers are stand-in addresses that are never dereferenced), and
the binding turns away tensors it cannot describe."""
import ctypes

import pytest

from gpu_util import ensure_built

P = 0x10000


@pytest.fixture(scope="module")
def abi():
    ensure_built()
    from gated_delta_rule_varlen_amd import _abi

    _abi.lib()
    return _abi


def attn_desc(abi, **f):
    base = dict(B=2, N=8, H=8, HK=2, D=64, max_q=6, dtype=1, flags=0, scale=0.0, prefix_len=0, kv_rows=100,
                q_stride=(512, 64), k_stride=(128, 64), v_stride=(128, 64), out_stride=(512, 64),
                prefix_k_stride=(128, 64), prefix_v_stride=(128, 64))
    base.update(f)
    return abi.AttnDesc(*[base[n] for n, _ in abi.AttnDesc._fields_])


def attention(abi, d, q=P, k=P, v=P, off=P, begin=P, length=P, out=P, lse=None, ws=P, ws_bytes=1 << 40):
    return abi.lib().gdn_attention_varlen(ctypes.byref(d), q, k, v, off, begin, length, out, lse, ws, ws_bytes, None, None)


@pytest.mark.parametrize(
    "fields,kw,want",
    [
        (dict(B=0), {}, "ERR_SHAPE"),
        (dict(N=-1), {}, "ERR_SHAPE"),
        (dict(H=0), {}, "ERR_SHAPE"),
        (dict(HK=0), {}, "ERR_SHAPE"),
        (dict(HK=3), {}, "ERR_SHAPE"),
        (dict(D=0), {}, "ERR_SHAPE"),
        (dict(D=264), {}, "ERR_SHAPE"),
        (dict(max_q=0), {}, "ERR_SHAPE"),
        (dict(kv_rows=-1), {}, "ERR_SHAPE"),
        (dict(prefix_len=-1), {}, "ERR_SHAPE"),
        (dict(prefix_len=5), {}, "ERR_SHAPE"),  # a prefix belongs to the other entry point
        (dict(scale=float("nan")), {}, "ERR_SHAPE"),
        (dict(scale=float("inf")), {}, "ERR_SHAPE"),
        (dict(q_stride=(-512, 64)), {}, "ERR_SHAPE"),
        (dict(k_stride=(128, -64)), {}, "ERR_SHAPE"),
        (dict(dtype=3), {}, "ERR_DTYPE"),
        (dict(flags=1), {}, "ERR_UNSUPPORTED"),
        (dict(N=2**30), {}, "ERR_OVERFLOW"),
        (dict(B=2**30), {}, "ERR_OVERFLOW"),
        (dict(k_stride=(2**22, 64)), {}, "ERR_OVERFLOW"),  # rows 8 MiB apart
        (dict(v_stride=(2**22, 64)), {}, "ERR_OVERFLOW"),
        (dict(k_stride=(128, 2**61)), {}, "ERR_OVERFLOW"),
        (dict(kv_rows=2**62), {}, "ERR_OVERFLOW"),
        (dict(D=60), {}, "ERR_ALIGN"),  # 120 bytes
        (dict(q_stride=(516, 64)), {}, "ERR_ALIGN"),
        (dict(out_stride=(512, 68)), {}, "ERR_ALIGN"),
        ({}, dict(q=None), "ERR_NULL"),
        ({}, dict(k=None), "ERR_NULL"),
        ({}, dict(v=None), "ERR_NULL"),
        ({}, dict(out=None), "ERR_NULL"),
        ({}, dict(off=None), "ERR_NULL"),
        ({}, dict(begin=None), "ERR_NULL"),  # runs and lengths come together
        ({}, dict(length=None), "ERR_NULL"),
        ({}, dict(q=P + 8), "ERR_ALIGN"),
        ({}, dict(v=P + 2), "ERR_ALIGN"),
        ({}, dict(ws=P + 4), "ERR_ALIGN"),
    ],
)
def test_attention_refusals(abi, fields, kw, want):
    assert attention(abi, attn_desc(abi, **fields), **kw) == getattr(abi, want)


@pytest.mark.parametrize(
    "fields,kw,want",
    [
        (dict(), dict(pk=None), "ERR_NULL"),
        (dict(), dict(pv=None), "ERR_NULL"),
        (dict(), dict(pk=P + 8), "ERR_ALIGN"),
        (dict(prefix_v_stride=(129, 64)), {}, "ERR_ALIGN"),
        (dict(prefix_k_stride=(2**22, 64)), {}, "ERR_OVERFLOW"),
        (dict(prefix_k_stride=(-128, 64)), {}, "ERR_SHAPE"),
    ],
)
def test_prefix_refusals(abi, fields, kw, want):
    d = attn_desc(abi, prefix_len=50, **fields)
    pk, pv = kw.get("pk", P), kw.get("pv", P)
    assert abi.lib().gdn_attention_prefix_varlen(ctypes.byref(d), P, pk, pv, P, P, P, P, P, P, None, P, 1 << 40, None,
                                                 None) == getattr(abi, want)


def test_missing_descriptors(abi):
    L = abi.lib()
    n = ctypes.c_size_t(0)
    assert L.gdn_attention_varlen(None, *([P] * 9), 0, None, None) == abi.ERR_NULL
    assert L.gdn_attention_prefix_varlen(None, *([P] * 11), 0, None, None) == abi.ERR_NULL
    assert L.gdn_qk_norm_rope_varlen(None, *([P] * 15)) == abi.ERR_NULL
    assert L.gdn_attention_workspace_bytes(None, ctypes.byref(n)) == abi.ERR_NULL
    assert L.gdn_attention_workspace_bytes(ctypes.byref(attn_desc(abi)), None) == abi.ERR_NULL


@pytest.mark.parametrize("fields", [{}, dict(prefix_len=4096), dict(N=256, B=256, max_q=1, kv_rows=1 << 20),
                                    dict(N=1, B=1, max_q=1, kv_rows=1 << 20), dict(N=0, max_q=0), dict(kv_rows=0)])
def test_workspace_is_what_the_call_asks_for(abi, fields):
    n = ctypes.c_size_t(1)
    d = attn_desc(abi, **fields)
    assert abi.lib().gdn_attention_workspace_bytes(ctypes.byref(d), ctypes.byref(n)) == abi.OK
    if n.value:
        args = [ctypes.byref(d), P, P, P, P, P, P, P, P, P, None]
        f = abi.lib().gdn_attention_prefix_varlen
        assert f(*args, P, n.value - 1, None, None) == abi.ERR_WORKSPACE
        assert f(*args, None, n.value, None, None) == abi.ERR_WORKSPACE


def rope_desc(abi, **f):
    base = dict(B=2, N=8, H=8, HK=2, D=64, rot=64, dtype=1, flags=0, eps=1e-6, reserved=0, cache_rows=100,
                q_stride=(512, 64), k_stride=(128, 64), v_stride=(128, 64), q_out_stride=(512, 64),
                k_out_stride=(128, 64), v_out_stride=(128, 64))
    base.update(f)
    return abi.RopeDesc(*[base[n] for n, _ in abi.RopeDesc._fields_])


@pytest.mark.parametrize(
    "fields,kw,want",
    [
        (dict(B=0), {}, "ERR_SHAPE"),
        (dict(N=-1), {}, "ERR_SHAPE"),
        (dict(H=0), {}, "ERR_SHAPE"),
        (dict(HK=0), {}, "ERR_SHAPE"),
        (dict(D=264), {}, "ERR_SHAPE"),
        (dict(rot=66), {}, "ERR_SHAPE"),
        (dict(rot=63), {}, "ERR_SHAPE"),
        (dict(rot=-2), {}, "ERR_SHAPE"),
        (dict(eps=-1.0), {}, "ERR_SHAPE"),
        (dict(eps=float("nan")), {}, "ERR_SHAPE"),
        (dict(cache_rows=-1), {}, "ERR_SHAPE"),
        (dict(reserved=1), {}, "ERR_SHAPE"),
        (dict(k_out_stride=(-128, 64)), {}, "ERR_SHAPE"),
        (dict(cache_rows=7), dict(begin=None), "ERR_SHAPE"),  # packed rows need one row per token
        (dict(dtype=9), {}, "ERR_DTYPE"),
        (dict(flags=2), {}, "ERR_UNSUPPORTED"),
        (dict(N=2**30), {}, "ERR_OVERFLOW"),
        (dict(N=2**30, H=1, HK=4), {}, "ERR_OVERFLOW"),
        (dict(k_out_stride=(2**60, 64)), {}, "ERR_OVERFLOW"),
        (dict(D=60, rot=60), {}, "ERR_ALIGN"),
        (dict(q_stride=(515, 64)), {}, "ERR_ALIGN"),
        ({}, dict(q=None), "ERR_NULL"),
        ({}, dict(k=None), "ERR_NULL"),
        ({}, dict(v=None), "ERR_NULL"),  # v and v_out come together
        ({}, dict(v_out=None), "ERR_NULL"),
        ({}, dict(k_out=None), "ERR_NULL"),
        ({}, dict(q_out=None), "ERR_NULL"),
        ({}, dict(freq=None), "ERR_NULL"),
        ({}, dict(off=None), "ERR_NULL"),
        ({}, dict(q=P + 8), "ERR_ALIGN"),
        ({}, dict(k_out=P + 4), "ERR_ALIGN"),
        ({}, dict(qw=P + 4), "ERR_ALIGN"),
    ],
)
def test_rope_refusals(abi, fields, kw, want):
    a = dict(q=P, k=P, v=P, freq=P, qw=P, kw=P, off=P, past=P, pos=P, begin=P, q_out=P, k_out=P, v_out=P)
    a.update(kw)
    d = rope_desc(abi, **fields)
    assert abi.lib().gdn_qk_norm_rope_varlen(ctypes.byref(d), *a.values(), None, None) == getattr(abi, want)


def test_the_binding_takes_device_tensors_only(abi):
    import torch

    import gated_delta_rule_varlen_amd as gdn

    x, off = torch.zeros(4, 2, 64), torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="device"):
        gdn.attention_varlen(x, x, x, off)
    with pytest.raises(ValueError, match="device"):
        gdn.attention_prefix_varlen(x, x, x, x, x, off)
    with pytest.raises(ValueError, match="device"):
        gdn.qk_norm_rope_varlen(x, x, x, off, inv_freq=torch.ones(32))
    with pytest.raises(ValueError, match="heads"):
        gdn.attention_varlen(x.view(4, 128), x, x, off)

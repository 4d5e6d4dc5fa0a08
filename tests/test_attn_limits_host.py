"""Refusals of lengths past what the attention's index arithmetic holds, on the host."""
import pytest

from test_attn_host import P, abi, attn_desc, attention, rope_desc  # noqa: F401


@pytest.mark.parametrize("prefix_len", [2**31 - 1, 2**31 - 4096])
def test_prefix_past_the_last_index(abi, prefix_len):  # noqa: F811
    import ctypes

    d = attn_desc(abi, prefix_len=prefix_len)
    n = ctypes.c_size_t()
    assert abi.lib().gdn_attention_workspace_bytes(ctypes.byref(d), ctypes.byref(n)) == abi.ERR_OVERFLOW
    assert abi.lib().gdn_attention_prefix_varlen(ctypes.byref(d), P, P, P, P, P, P, P, P, P, None, P, 1 << 40, None,
                                                 None) == abi.ERR_OVERFLOW


@pytest.mark.parametrize("bad", ["q", "k", "offsets"])
def test_the_binding_takes_tensors_only(abi, bad):  # noqa: F811
    import torch

    import gated_delta_rule_varlen_amd as gdn

    x = dict(q=torch.zeros(4, 2, 64), k=torch.zeros(4, 2, 64), v=torch.zeros(4, 2, 64),
             offsets=torch.tensor([0, 4], dtype=torch.int32))
    x[bad] = 3
    with pytest.raises((TypeError, ValueError)):
        gdn.attention_varlen(*x.values())
    with pytest.raises((TypeError, ValueError)):
        gdn.qk_norm_rope_varlen(*x.values(), inv_freq=torch.ones(32))
    with pytest.raises((TypeError, ValueError)):
        gdn.attention_prefix_varlen(x["q"], None, None, x["k"], x["v"], x["offsets"])


@pytest.mark.parametrize("call", ["eps", "scale", "max_q"])
def test_numbers_that_are_none(abi, call):  # noqa: F811
    import torch

    import gated_delta_rule_varlen_amd as gdn

    x, off = torch.zeros(4, 2, 64), torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises((TypeError, ValueError)):
        if call == "eps":
            gdn.qk_norm_rope_varlen(x, x, x, off, inv_freq=torch.ones(32), eps="small")
        else:
            gdn.attention_varlen(x, x, x, off, **{call: "one"})


@pytest.mark.parametrize("fields", [dict(N=2**31 - 100, H=1, HK=1), dict(N=(2**31 - 1) // 16, H=16, HK=1)])
def test_rows_past_the_last_index(abi, fields):  # noqa: F811
    """A row tile past the last row still has an index of 32 bits."""
    import ctypes

    n = ctypes.c_size_t()
    for max_q in (1, fields["N"]):
        d = attn_desc(abi, **fields, max_q=max_q)
        assert attention(abi, d) == abi.ERR_OVERFLOW
        assert abi.lib().gdn_attention_workspace_bytes(ctypes.byref(d), ctypes.byref(n)) == abi.ERR_OVERFLOW


@pytest.mark.parametrize("N", [2**31 - 1, 2**31 - 4096])
def test_tokens_past_the_last_index(abi, N):  # noqa: F811
    import ctypes

    d = rope_desc(abi, N=N, H=1, HK=1, cache_rows=N)
    assert abi.lib().gdn_qk_norm_rope_varlen(ctypes.byref(d), *([P] * 13), None, None) == abi.ERR_OVERFLOW


@pytest.mark.parametrize("fields", [dict(B=2**24, N=2**10, max_q=2**10), dict(B=2**27, N=2**7, max_q=2**7)])
def test_more_row_tiles_than_a_launch_holds(abi, fields):  # noqa: F811
    assert attention(abi, attn_desc(abi, **fields)) == abi.ERR_OVERFLOW


@pytest.mark.parametrize("N", [2**26, 2**30])
def test_more_tokens_than_a_launch_holds(abi, N):  # noqa: F811
    import ctypes

    for rot in (64, 50):
        d = rope_desc(abi, N=N, H=1, HK=1, cache_rows=N, rot=rot)
        assert abi.lib().gdn_qk_norm_rope_varlen(ctypes.byref(d), *([P] * 13), None, None) == abi.ERR_OVERFLOW


@pytest.mark.parametrize("fields,rows", [(dict(H=16, HK=2, D=256, max_q=4), 32), (dict(H=8, HK=2, D=128, max_q=16), 64),
                                         (dict(H=8, HK=2, D=128, max_q=16, dtype=0), 64)])
def test_two_blocks_a_cu_where_they_fit(abi, fields, rows):  # noqa: F811
    """Rings and queries of exactly half a CU's LDS (80 KB): the workspace has slots for two blocks on each of 256
    CUs.  At fp32 and D 128 the 64 rows leave one."""
    import ctypes

    n = ctypes.c_size_t()
    D, H = fields["D"], fields["H"]
    wide = dict(q_stride=(H * D, D), out_stride=(H * D, D), k_stride=(2 * D, D), v_stride=(2 * D, D))
    d = attn_desc(abi, B=64, N=64 * fields["max_q"], kv_rows=1 << 20, **fields, **wide)
    assert abi.lib().gdn_attention_workspace_bytes(ctypes.byref(d), ctypes.byref(n)) == abi.OK
    blocks = 256 if fields.get("dtype") == 0 else 512
    slots = 2 * blocks * rows * (4 * D + 8)
    assert slots <= n.value < slots + slots // 8

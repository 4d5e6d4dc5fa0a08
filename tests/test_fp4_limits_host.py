"""Limits of the 4-bit cache's write and read on the host: a token's elements are counted in 32 bits."""
import pytest

from test_fp4_host import abi, cache_of, rows_call  # noqa: F401


@pytest.mark.parametrize("read", [False, True])
@pytest.mark.parametrize("HK,D", [(2**26, 256), (2**23, 256), (2**26 - 128, 32), (2**29, 128)])
def test_tokens_of_too_many_elements(abi, read, HK, D):  # noqa: F811
    cache = cache_of(abi, **{f"{x}_{y}_stride": (16, 16) if y == "codes" else (0, 8) for x in "kv" for y in ("codes", "scales")})
    fields = dict(B=1, N=1, HK=HK, D=D, k_stride=(0, D), v_stride=(0, D))
    assert rows_call(abi, read, fields, cache) == abi.ERR_OVERFLOW

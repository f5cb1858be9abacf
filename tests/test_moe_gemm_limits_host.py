"""Extents of the 8-bit product next to 2^31, whose rounding up to tiles would leave
32 bits: refused on the host (no GPU; run where there is none)."""
import pytest

from test_moe_ops_host import GEMM, abi  # noqa: F401


@pytest.mark.parametrize("over", [
    dict(rows=2 ** 31 - 1), dict(rows=2 ** 31 - 256), dict(rows=2 ** 31 - 2 ** 23),
    dict(N=2 ** 31 - 1), dict(N=2 ** 31 - 128), dict(N=2 ** 31 - 255),
    dict(hidden=2 ** 31 - 16), dict(hidden=2 ** 31 - 112),
    dict(groups=127, rows=16909320), dict(groups=127, N=16909320)])
def test_extents_next_to_the_limit_are_refused(abi, over):  # noqa: F811
    args = {**GEMM, "groups": 1, "rows": 1, "N": 1, **over}
    assert abi.moe_gemm_int8(**args) == abi.MOE_ERR_INVALID_ARG

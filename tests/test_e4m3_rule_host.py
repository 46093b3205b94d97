"""Which form of the 8-bit products a call takes, by its sizes and its result's type."""
import os

import pytest

import causal_gqa_attention_rmsnorm_gb300 as tb
from causal_gqa_attention_rmsnorm_gb300 import binding


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        pytest.skip("libtb.so not built")
    return binding.lib()


# K up to which one accumulator holds all of a sum
@pytest.mark.parametrize("dtype,K", [(tb.TB_F32, 4096), (tb.TB_BF16, 65536), (tb.TB_E4M3, 65536)])
@pytest.mark.parametrize("mats", [1, 2])
@pytest.mark.parametrize("M", [100, 8192])
def test_long_sums_are_formed_in_parts(lib, M, mats, dtype, K):
    if mats == 1 and dtype == tb.TB_E4M3:
        return                                          # (a product's result is no codes)
    N = 65536
    for res in (0, 1):
        assert lib.tbx_e4m3_tile(M, N, K, mats, dtype, res, 152) == (0 if M > 128 else -1)
        assert lib.tbx_e4m3_tile(M, N, K + 16, mats, dtype, res, 152) == (128 if mats == 1 else 64)
        assert lib.tbx_e4m3_tile(M, N, 2 ** 31 - 1024, mats, dtype, res, 152) > 0
    # what the small tiles have anyway they keep
    for k in (K, K + 16):
        assert lib.tbx_e4m3_tile(9, N, k, mats, dtype, 0, 152) == 16

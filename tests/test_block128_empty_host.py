"""Calls with nothing to compute need no memory (an empty tensor's address is null)."""
import pytest
import torch

import block_scaled_fp8_sm_gb300 as bs
from block_scaled_fp8_sm_gb300 import _abi


@pytest.fixture(scope="module")
def lib():
    from block_scaled_fp8_sm_gb300 import build
    build.build()
    return bs.library()


@pytest.mark.parametrize("T,N,K,E", [(64, 64, 64, 0), (0, 64, 64, 4), (64, 0, 64, 4), (0, 0, 0, 0), (64, 64, 0, 0)])
def test_experts(lib, T, N, K, E):
    for mode in (0, 1, 2):
        assert lib.fp8_gemm_experts_ex(0, 0, 0, 0, 0, 0, T, N, K, E, mode, None) == _abi.FP8_OK
    assert lib.fp8_gemm_experts_ex(0, 0, 0, 0, 0, 0, T, N, K, E, 5, None) == _abi.FP8_ERR_MODE


@pytest.mark.parametrize("bad", [(64, 60, 64), (64, 64, 24), (-1, 64, 64), (64, 64, 1 << 30)])
def test_without_experts_the_sizes_are_checked(lib, bad):
    assert lib.fp8_gemm_experts_ex(0, 0, 0, 0, 0, 0, *bad, 0, 0, None) == _abi.FP8_ERR_SHAPE


def test_an_empty_tensor_is_a_null_pointer():
    assert torch.empty(0, 64, 64, dtype=torch.uint8).data_ptr() == 0

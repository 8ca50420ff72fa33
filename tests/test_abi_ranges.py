"""Sizes whose launches would have 2^32 threads and more along an axis, which the
runtime drops without an error, are refused before."""

import os

import pytest

from fp8_block_scaled_quant_amd import _lib

P = 4096   # never dereferenced
COLS = 80 * ((1 << 22) - 1) + 1
WIDE = 128 * ((1 << 24) - 1) + 1


@pytest.fixture(scope="module")
def lib():
    return _lib.load_library(os.environ.get("FP8BSQ_TEST_LIB"))


@pytest.mark.parametrize("m", [1, 40, 300])
def test_products(lib, m):
    for name in ("fp8_block_gemm", "fp8_block_gemm_ue8m0", "fp8_block_gemm_reference"):
        assert getattr(lib, name)(P, P, P, P, P, 1, m, COLS, 128, None) == _lib.ERANGE
    assert lib.fp8_block_gemm_split_workspace(m, COLS, 128) == 0
    assert lib.fp8_block_gemm_split(P, P, P, P, P, 1, m, COLS, 128, 0, P, 1 << 40, None) == _lib.ERANGE
    assert lib.fp8_block_gemm_split_noalloc(P, P, P, P, P, 1, m, COLS, 128, 0, None) == _lib.ERANGE
    assert lib.fp8_act_quant_gemm(P, 1, 0, P, P, None, P, 1, m, COLS, 128, P, P, None) == _lib.ERANGE


def test_weights(lib):
    assert lib.fp8_weight_quant(P, 1, 1, WIDE, 128, 0, P, P, None) == _lib.ERANGE
    assert lib.fp8_weight_dequant(P, P, 1, WIDE, 128, P, 1, None) == _lib.ERANGE

"""Sizes beyond the ranges of the feed-forward entry points: the status says so
whatever workspace comes with them, as the workspace functions answer 0 there."""

import pytest

from fp8_block_scaled_quant_amd import _ffn_lib, _lib

P = 4096   # never dereferenced


@pytest.fixture(scope="module")
def lib():
    return _ffn_lib.load_library()


@pytest.mark.parametrize("workspace", [None, P])
@pytest.mark.parametrize("m,f,k", [(65535 * 16 + 1, 128, 128), (1, (1 << 21) + 128, 128), (1, 128, (1 << 21) + 128)])
def test_products_out_of_range(lib, m, f, k, workspace):
    assert lib.fp8_gated_ffn_workspace(m, f, k) == 0 and lib.fp8_gated_ffn_backward_workspace(m, f, k) == 0
    assert lib.fp8_gated_ffn(P, 1, 0, P, P, P, P, P, None, None, 1, m, f, k, workspace, 0, None) == _lib.ERANGE
    assert lib.fp8_gated_ffn_backward(P, P, P, P, 1, P, P, P, P, P, P, P, 1, m, f, k, workspace, 0, None) == _lib.ERANGE


def test_missing_and_small_workspaces_within_range(lib):
    for workspace, status in ((None, _lib.EINVAL), (P, _lib.ESCRATCH)):
        assert lib.fp8_gated_ffn(P, 1, 0, P, P, P, P, P, None, None, 1, 40, 128, 128, workspace, 0, None) == status
        assert lib.fp8_gated_ffn_backward(P, P, P, P, 1, P, P, P, P, P, P, P, 1, 40, 128, 128, workspace, 0, None) == status


def test_fp4_gemv_out_of_range(lib):
    """A weight row more than the threads of one launch reach."""
    for m, n, k in ((1, 144 * ((1 << 22) - 1) + 1, 32), (65535 * 16 + 1, 8, 32), (1, 8, (1 << 27) + 32)):
        assert lib.fp4_gemv(P, 1, P, P, None, P, 1, m, n, k, None) == _lib.ERANGE

"""Sizes that the matrix product of scaled 8-bit matrices takes, up to its
limits: host-side checks, without a GPU."""
import ctypes

import pytest

from test_fp8_abi import UNSUPPORTED, WORKSPACE, _mm, lib  # noqa: F401

M = (1 << 31) - 1025  # the largest size; a missing workspace is found after the sizes


@pytest.mark.parametrize("kw,want", [
    (dict(m=M, n=1, ldo=1), WORKSPACE), (dict(m=M + 1, n=1, ldo=1), UNSUPPORTED),
    (dict(m=1, n=M, ldo=M), WORKSPACE), (dict(m=1, n=M + 1, ldo=M + 1), UNSUPPORTED),
    (dict(k=M, lda=M + 1, ldb=M + 1), WORKSPACE), (dict(k=M + 1, lda=M + 1, ldb=M + 1), UNSUPPORTED),
    (dict(lda=(1 << 31) - 16), WORKSPACE), (dict(lda=1 << 31), UNSUPPORTED),
    (dict(ldb=(1 << 31) - 16), WORKSPACE), (dict(ldb=1 << 31), UNSUPPORTED),
    # 2^25 - 1 = 31 x 1082401 blocks, and 2^25
    (dict(m=31 * 128, n=1082401 * 128, ldo=1082401 * 128), WORKSPACE),
    (dict(m=1 << 18, n=1 << 21, ldo=1 << 21), UNSUPPORTED)])
def test_matmul_takes_sizes_up_to_its_limits(lib, kw, want):  # noqa: F811
    assert lib.kda_fp8_matmul(ctypes.byref(_mm(workspace=None, **kw)), None) == want

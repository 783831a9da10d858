"""CPU tests of what the calls of include/sparse_ffn_experts.h refuse, or split up, at their
largest sizes: nothing is launched here."""
import ctypes as C
import os
import subprocess

import pytest

from test_experts_abi import A, N, desc, experts, matmul  # noqa: F401

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
MOST = (1 << 31) - 1


def test_channels_and_columns_near_32_bits_are_refused(N):  # noqa: F811
    """Tiles round channels, and rows of 16 bytes columns, up in 32 bits."""
    for n in (MOST, MOST - 100, MOST - 1022):
        assert matmul(N, N=n, ldy=n) == N.SFFN_ERR_UNSUPPORTED
        assert matmul(N, N=n, ldy=n, M=1, work=None, work_bytes=0) == N.SFFN_ERR_UNSUPPORTED
        a = dict(x=A, dtype=1, ldx=n, rows=1, cols=n, q=A, ldq=1 << 31, scale=A, stream=None)
        assert N.lib().sparse_ffn_quantize_rows(*a.values()) == N.SFFN_ERR_UNSUPPORTED


def test_products_past_one_launch_are_refused(N):  # noqa: F811
    """A launch holds less than 2^32 threads: 2^24 tiles of 64 rows x 128 channels are too many."""
    for M in (65, 96):
        assert matmul(N, M=M, N=1 << 30, ldy=1 << 30) == N.SFFN_ERR_UNSUPPORTED
    assert matmul(N, M=1 << 20, N=1 << 20, ldy=1 << 20) == N.SFFN_ERR_UNSUPPORTED

"""CPU tests of the fp8 products' limits: what a kernel could not be launched for is refused
before any device access; nothing else is."""
import os

import pytest

from bit_quantized_linear_rotate_amd import _binding as b

pytestmark = pytest.mark.skipif(not os.path.exists(b.LIB_PATH), reason="libw4a4.so not built")

P = 0x1000   # an aligned pointer that nothing reads: every call ends in validation


def gemm(M, K, N):
    return b.lib().w8a8_gemm_fp8(P, P, M, K, P, P, N, None, 0, P, 2, None)


def grouped(M, K, E, N, R):
    return b.lib().w8a8_grouped_gemm_fp8(P, P, M, K, P, P, E, N, P, P, R, None, 0, P, 2, None)


def test_more_threads_than_a_launch_has_are_refused():
    # the skinny kernel: a workgroup of 512 threads to 32 columns, 2^32 - 512 threads at most
    assert gemm(1, 1040, 1 << 28) == b.UNSUPPORTED
    assert gemm(64, 1040, (1 << 28) - 31) == b.UNSUPPORTED


def test_tiles_beyond_31_bits_are_refused():
    assert gemm(1 << 28, 16, 1 << 16) == b.UNSUPPORTED
    assert grouped(4, 16, 2, 1 << 20, 1 << 30) == b.UNSUPPORTED

"""CPU tests of further refusals of the MX4 entry points, by the binding (ValueError) and
by the C ABI (status codes), before any device access; and of host-only choices."""
import os

import pytest
import torch

from bit_quantized_linear_rotate_amd import _binding as b
from tests.test_mx4_refusals import BF, E, FAKE, K, M, N, args, z

pytestmark = pytest.mark.skipif(not os.path.exists(b.LIB_PATH), reason="libw4a4.so not built")


def test_row_types_are_refused():
    with pytest.raises(ValueError, match="rows_dtype"):
        b.w4a4_experts_mx4(**args("w4a4_experts_mx4", rows_dtype=torch.float16))
    for over in (dict(out_dtype=torch.float32), dict(y=torch.zeros(M, N), out_dtype=torch.float64)):
        with pytest.raises(ValueError, match="out_dtype"):
            b.w4a4_combine_experts(**args("w4a4_combine_experts", **over))
    with pytest.raises(ValueError, match="CUDA"):
        b.w4a4_experts_mx4(**args("w4a4_experts_mx4", rows_dtype=torch.float32))
    L = b.lib()
    to = lambda dt, od: L.w4a4_combine_experts_to(FAKE, dt, 4, 8, FAKE, FAKE, 4, 2, FAKE, od, None)  # noqa: E731
    assert to(2, 0) == b.UNSUPPORTED and to(0, 5) == b.UNSUPPORTED and to(7, 7) == b.UNSUPPORTED
    rows = lambda dt, need: L.w4a4_experts_mx4_rows(  # noqa: E731
        FAKE, 2, M, K, K, 1, 0, None, None, FAKE, 0, E, E, 2, 1, FAKE, FAKE, 64, FAKE, FAKE, dt, FAKE, FAKE, need, None)
    assert rows(1, 1 << 30) == b.UNSUPPORTED and rows(9, 1 << 30) == b.UNSUPPORTED
    small = b.w4a4_experts_mx4_workspace_size(M, K, 64, E, 2, BF)
    need = b.w4a4_experts_mx4_workspace_size(M, K, 64, E, 2, torch.float32)
    assert need > small and rows(0, need - 1) == b.INVALID and b"workspace" in L.w4a4_last_error()


def test_token_counts_past_any_memory_are_refused():
    L = b.lib()
    for T, k in ((1 << 62, 4), (1 << 61, 8), (1 << 31, 1), (1 << 30, 2)):
        rc = L.w4a4_route_experts(FAKE, 0, T, 8, 8, k, 1, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 30, None)
        assert rc == b.UNSUPPORTED and b"top_k" in L.w4a4_last_error()


def test_one_row_of_one_expert_is_the_skinny_kernels():
    """However narrow the output: a tile of 64 x 256 is never cheaper than 16 columns a wave."""
    for K in (512, 1824, 3840):
        for n in (64, 96, 256):
            for experts in (0, 1, 2):
                assert b.w4a4_gemm_mx4_plan(1, K, n, experts) == "skinny", (K, n, experts)
            assert b.w4a4_gemm_mx4_plan(1, K, n, 1, True) == "skinny", (K, n)

"""GPU tests of grouped products whose first offset is not zero (a slice of a longer
list of experts): the sorted rows before it belong to nobody and come back as zeros,
like those past the last offset, whatever the output held before."""
import numpy as np
import pytest
import torch

from tests import mx4
from tests.gpu_util import need_gpu
from tests.test_gpu_mx4 import DT, as64, operand

pytestmark = pytest.mark.gpu

import bit_quantized_linear_rotate_amd as w4  # noqa: E402
from bit_quantized_linear_rotate_amd import _binding as b  # noqa: E402

# rows before the first expert, of each expert, and past the last; the kernel taken
CASES = [(3, [5, 0, 2], 4, 256, 192, "skinny"), (70, [0, 0], 3, 96, 192, "skinny"),
         (37, [200, 0, 150], 5, 512, 256, "tile64"), (261, [700, 1, 900, 333, 0, 513, 64], 9, 288, 2304, "tile128"),
         (300, [2600, 1, 2049, 513], 0, 1056, 2368, "tile256")]


def stream():
    return torch.cuda.current_stream().cuda_stream


@pytest.mark.parametrize("case", CASES, ids=lambda c: c[-1])
@pytest.mark.parametrize("out", ["f32", "bf16"])
def test_rows_before_the_first_expert(case, out):
    need_gpu()
    before, counts, after, K, N, kernel = case
    E, R = len(counts), before + sum(counts) + after
    a, sa, av = operand(R, K, 1)
    w, sw, wv = operand(N, K, 2, (E,))
    off = torch.from_numpy((before + np.concatenate([[0], np.cumsum(counts)])).astype(np.int32)).cuda()
    o = off.cpu().numpy()
    assert w4.w4a4_gemm_mx4_plan(R, K, N, E) == w4.w4a4_gemm_mx4_plan(R, K, N, E, True) == kernel
    got = torch.full((R, N), 7.0, dtype=DT[out], device="cuda")
    rc = b.lib().w4a4_grouped_gemm_mx4(a.data_ptr(), sa.data_ptr(), R, K, w.data_ptr(), sw.data_ptr(), E, N,
                                       off.data_ptr(), None, R, None, 0, got.data_ptr(), b._DT[DT[out]], stream())
    assert rc == b.OK
    ref, bound = np.zeros((R, N)), np.zeros((R, N))
    for e in range(E):
        at = slice(o[e], o[e + 1])
        ref[at], bound[at] = av[at] @ wv[e].T, mx4.product_bound(av[at], wv[e])
    mx4.close(as64(got), ref, bound, out)
    assert bool((got[:before] == 0).all()) and bool((got[o[E]:] == 0).all())
    # gated: codes and scales of the same rows
    F = N // 2
    codes = torch.full((R, F // 2), 0xAB, dtype=torch.uint8, device="cuda")
    scales = torch.full((-(-F // 256), R, 8), 0xAB, dtype=torch.uint8, device="cuda")
    rc = b.lib().w4a4_grouped_gated_mx4(a.data_ptr(), sa.data_ptr(), R, K, w.data_ptr(), sw.data_ptr(), E, N,
                                        off.data_ptr(), None, R, None, 0, codes.data_ptr(), scales.data_ptr(), stream())
    assert rc == b.OK
    for at in (slice(0, before), slice(o[E], R)):
        assert not bool(codes[at].any()) and not bool(scales[:, at].any())
    # the experts' rows as in a list of their own, where that takes the same kernel
    if sum(counts) and w4.w4a4_gemm_mx4_plan(sum(counts), K, N, E, True) == kernel:
        own = slice(before, int(o[E]))
        c, s = w4.w4a4_grouped_gated_mx4(a[own].contiguous(), sa[:, own].contiguous(), w, sw, off - before)
        assert torch.equal(c, codes[own]) and torch.equal(s, scales[:, own])

"""GPU tests of the expert layer whose experts' rows stay in single precision until
the weighted sum (rows_dtype), against 64 bits."""
import numpy as np
import pytest
import torch

from tests import mx4
from tests.gpu_util import need_gpu
from tests.test_gpu_mx4 import DT, as64, draw_x, operand, signs
from tests.test_gpu_mx4_experts import logits_of

pytestmark = pytest.mark.gpu

import bit_quantized_linear_rotate_amd as w4  # noqa: E402


@pytest.mark.parametrize("T,E,k", [(1, 4, 2), (16, 32, 4), (300, 8, 2), (700, 6, 3)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_layer_rounds_once(T, E, k, dtype):
    """Against 64 bits from the codes of the hidden rows: the fp32 sums' error and one
    rounding, with nothing for the rows between; and the layer is its parts."""
    need_gpu()
    K, F, g = 512, 288, 64
    _, sid = signs(g, 3)
    h = w4.Hadamard(g, sid)
    x = draw_x(T, K, dtype, 1)
    l = logits_of(T, E, "f32", 2)
    w13, s13, _ = operand(2 * F, K, 3, (E,))
    w2, s2, v2 = operand(K, F, 4, (E,))
    s13 = (s13.int() - 6).clamp(min=0).to(torch.uint8)
    got = w4.w4a4_experts_mx4(x, l, k, w13, s13, w2, s2, h=h, rows_dtype=torch.float32)
    assert got.dtype == DT[dtype]
    weights, experts, rows, pos, off = w4.w4a4_route_experts(l, k)
    c, s = w4.w4a4_quantize_mx4(x, h)
    ac, as_ = w4.w4a4_grouped_gated_mx4(c, s, w13, s13, off, rows=rows)
    y = w4.w4a4_grouped_gemm_mx4(ac, as_, w2, s2, off, out_dtype=torch.float32)
    assert torch.equal(got, w4.w4a4_combine_experts(y, pos, weights, out_dtype=DT[dtype]))
    act = mx4.values(ac.cpu().numpy(), mx4.unslab(as_.cpu().numpy(), F))
    o, p, wt = off.cpu().numpy(), pos.cpu().numpy(), as64(weights)
    yy, bound = np.zeros((T * k, K)), np.zeros((T * k, K))
    for e in range(E):
        at = slice(o[e], o[e + 1])
        yy[at] = act[at] @ v2[e].T
        bound[at] = mx4.product_bound(act[at], v2[e])
    each = lambda v: (np.where((p >= 0)[..., None], v[np.maximum(p, 0)], 0) * wt[..., None]).sum(1)  # noqa: E731
    mx4.close(as64(got), each(yy), each(bound) + (k + 1) * 2.0 ** -24 * each(np.abs(yy)), dtype)
    # a workspace of the size asked for, and one that is too small
    need = w4.w4a4_experts_mx4_workspace_size(T, K, F, E, k, torch.float32)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    again = w4.w4a4_experts_mx4(x, l, k, w13, s13, w2, s2, h=h, rows_dtype=torch.float32, workspace=ws)
    assert torch.equal(again, got)
    with pytest.raises(ValueError, match="workspace"):
        w4.w4a4_experts_mx4(x, l, k, w13, s13, w2, s2, h=h, rows_dtype=torch.float32, workspace=ws[:-1])


@pytest.mark.parametrize("out", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("T,k,N", [(1, 1, 1), (3, 4, 77), (70, 8, 256), (513, 3, 2052)])
def test_combine_fp32_rows(T, k, N, out):
    need_gpu()
    r = np.random.default_rng(T)
    R = max(1, T * k - 2)
    y = torch.randn(R, N, device="cuda")
    pos = r.integers(-1, R, (T, k)).astype(np.int32)
    pos[0] = -1
    w = torch.rand(T, k, device="cuda")
    p = torch.from_numpy(pos).cuda()
    got = w4.w4a4_combine_experts(y, p, w, out_dtype=DT[out])
    assert torch.equal(got, w4.w4a4_combine_experts(y, p, w).to(DT[out]))     # rounded once, to nearest
    v = np.where((pos >= 0)[..., None], as64(y)[np.maximum(pos, 0)], 0) * as64(w)[..., None]
    mx4.close(as64(got), v.sum(1), (k + 1) * 2.0 ** -24 * np.abs(v).sum(1), out)

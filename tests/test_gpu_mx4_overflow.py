"""GPU tests of rotated rows whose butterflies leave the range of fp32: every block that
ends with a NaN or an infinity is marked, bit for bit as the definition."""
import numpy as np
import pytest
import torch

from tests import mx4
from tests.gpu_util import need_gpu
from tests.test_gpu_mx4 import DT, check_quantized, signs

pytestmark = pytest.mark.gpu

import bit_quantized_linear_rotate_amd as w4  # noqa: E402


def rows_of(g):
    """Finite rows of 512 whose sums of up to g values overflow: in one butterfly, in
    all, with infinities that cancel to a NaN beside finite values."""
    r = np.random.default_rng(g)
    K = 512
    x = []
    for v in (6e37, 2e37, 2.0 ** 123, 2.0 ** 126):
        x.append(np.full(K, v))
        for n in (8, 32):                                  # the last n of each group of four times as many negative
            x.append(np.where(np.arange(K) % (4 * n) < 3 * n, v, -v))
    for lo, hi in ((120, 124), (122, 127), (126, 127.9)):
        x += list(np.exp2(r.uniform(lo, hi, (4, K))) * r.choice([-1, 1], (4, K)))
    one = np.zeros(K)                                      # few values, zeros elsewhere
    one[[0, 1, 32, 33, 64, 96]] = 2e38
    x += [one, np.roll(one, 16), -one, r.standard_normal(K)]
    return torch.from_numpy(np.stack(x))


@pytest.mark.filterwarnings("ignore:overflow:RuntimeWarning")
@pytest.mark.filterwarnings("ignore:invalid value:RuntimeWarning")
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("g", [16, 32, 64, 128, 256])
def test_overflow_in_the_rotation(g, dtype):
    need_gpu()
    x = rows_of(g).to(DT[dtype])
    assert bool(torch.isfinite(x).all())
    y = mx4.rotate(x.float().numpy(), g).reshape(len(x), -1, 32)
    if g > 16:   # the rows are what they are for: blocks whose only NaN stands beside finite values
        assert (np.isnan(y).any(-1) & np.isfinite(y).any(-1) & ~np.isinf(y).any(-1)).any()
    check_quantized(x.cuda(), w4.Hadamard(g), None, None)
    si, sid = signs(g, 1)
    so, sod = signs(g, 2)
    check_quantized(x.cuda(), w4.Hadamard(g, sid, sod), si, so)
    # the layer's rows are NaN there, and only there
    codes, scales = w4.w4a4_quantize_mx4(torch.eye(512, device="cuda").to(DT[dtype]))
    out = w4.w4a4_linear_mx4(x.cuda(), codes, scales, h=w4.Hadamard(g), out_dtype=torch.float32)
    bad = ~np.isfinite(y).all(-1)
    assert np.array_equal(np.isnan(out.cpu().numpy()).all(1), bad.any(1))

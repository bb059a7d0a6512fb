"""GPU tests of the MX4 quantiser, product and linear layer against plain forms in
64 bits (tests/mx4.py).  Codes and scales are compared bit for bit; products
against a bound on the fp32 sums plus one rounding to the output type."""
import numpy as np
import pytest
import torch

from tests import mx4
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu

import bit_quantized_linear_rotate_amd as w4  # noqa: E402

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def signs(g, seed):
    s = np.random.default_rng(seed).choice([-1, 1], g).astype(np.int8)
    return s, torch.from_numpy(s).cuda()


def as64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def draw_x(M, K, dtype, seed):
    """Rows with outliers, small rows, exact ties, zeros."""
    r = np.random.default_rng(seed)
    x = r.standard_normal((M, K)) * np.where(r.random(K) < 0.02, 20, 1)
    x[::7] *= 2.0 ** -9
    x[1::5] = np.round(x[1::5] * 4) / 4
    x[2::11] = 0
    return torch.from_numpy(x).to(DT[dtype]).cuda()


def check_quantized(x, h, sign_in, sign_out):
    codes, scales = w4.w4a4_quantize_mx4(x, h)
    M, K = x.shape
    y = x.detach().cpu().to(torch.float32).numpy()
    if h is not None:
        y = mx4.rotate(y, h.g, sign_in, sign_out)
    rc, rs = mx4.quantize(y)
    assert codes.shape == (M, K // 2) and scales.shape == (-(-K // 256), M, 8)
    assert np.array_equal(codes.cpu().numpy(), rc)
    assert np.array_equal(scales.cpu().numpy(), mx4.slabs(rs))
    return codes, scales, rc, rs


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,K", [(1, 32), (3, 96), (33, 256), (7, 288), (130, 1024), (5, 3840)])
def test_quantize_is_the_definition(M, K, dtype):
    need_gpu()
    x = draw_x(M, K, dtype, M + K)
    codes, scales, rc, rs = check_quantized(x, None, None, None)
    v = mx4.values(rc, rs)
    for out in DT:
        back = w4.w4a4_dequantize_mx4(codes, scales, DT[out])
        ref = torch.from_numpy(v).to(torch.float32).to(DT[out])
        assert torch.equal(back.cpu().float(), ref.float())


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("g", [16, 32, 64, 128, 256])
def test_quantize_rotated_is_the_definition(g, dtype):
    need_gpu()
    for M, K, seed in ((9, 3 * 256, 1), (70, 256, 2), (2, max(32, g), 3)):
        si, sid = signs(g, seed)
        so, sod = signs(g, seed + 10)
        x = draw_x(M, K, dtype, seed)
        check_quantized(x, w4.Hadamard(g, sid, sod), si, so)
        check_quantized(x, w4.Hadamard(g), None, None)


def test_quantize_many_rows_take_the_unrolled_kernel():
    need_gpu()
    for M in (8192 + 5, 32 * 1024):   # 257 and 1024 row groups of 32, several slabs
        x = draw_x(M, 1056, "bf16", M)
        si, sid = signs(32, 4)
        check_quantized(x, w4.Hadamard(32, sid), si, None)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_quantize_strides(dtype):
    need_gpu()
    x = draw_x(37, 512, dtype, 5)
    ref = w4.w4a4_quantize_mx4(x)
    wide = torch.zeros((37, 520 + 3), dtype=x.dtype, device="cuda")
    wide[:, 3:515] = x                                     # misaligned rows
    views = [x.t().contiguous().t(), wide[:, 3:515], torch.stack([x, x], 2)[:, :, 0]]
    for v in views:
        got = w4.w4a4_quantize_mx4(v)
        assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    got = w4.w4a4_quantize_mx4(x[5:6])
    assert torch.equal(got[0], ref[0][5:6]) and torch.equal(got[1], ref[1][:, 5:6])


def test_quantize_every_16bit_pattern():
    """Every bf16 and fp16 value at every position of the grid: as the only large value
    of its block, and beside a larger one."""
    need_gpu()
    for dtype in ("bf16", "f16"):
        bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
        v = bits.view(DT[dtype])
        v = v[torch.isfinite(v)]
        n = v.numel() // 32 * 32
        x = v[:n].reshape(-1, 32).cuda()                   # neighbouring patterns
        check_quantized(x, None, None, None)
        y = torch.zeros((v.numel(), 32), dtype=v.dtype)
        y[:, 0], y[:, 9] = v, v * 0.4375                   # a value and a smaller one
        check_quantized(y.cuda(), None, None, None)


def test_quantize_extremes():
    need_gpu()
    big, tiny = 3.3895313892515355e38, 2.0 ** -133
    x = torch.zeros((6, 64), dtype=torch.bfloat16)
    x[0, 3], x[0, 40] = big, -big
    x[1, :] = tiny
    x[2, 5] = -0.0
    x[3, 7] = float("nan")
    x[4, 33] = float("inf")
    x[5, 1], x[5, 2] = 2.0 ** -126, -(2.0 ** -130)
    check_quantized(x.cuda(), None, None, None)
    codes, scales = w4.w4a4_quantize_mx4(x.cuda())
    v = as64(w4.w4a4_dequantize_mx4(codes, scales, torch.float32))
    assert np.isnan(v[3, :32]).all() and not np.isnan(v[3, 32:]).any()
    assert np.isnan(v[4, 32:]).all() and not np.isnan(v[4, :32]).any()
    f = torch.tensor([[2.0 ** -149, -(2.0 ** -127), 3e-39] + [0.0] * 29, [float("nan")] * 32], dtype=torch.float32)
    check_quantized(f.cuda(), None, None, None)
    # rotation spreads a NaN over its group and no further
    x = torch.ones((1, 256), dtype=torch.float16)
    x[0, 70] = float("nan")
    codes, scales = w4.w4a4_quantize_mx4(x.cuda(), w4.Hadamard(64))
    v = as64(w4.w4a4_dequantize_mx4(codes, scales, torch.float32))
    assert np.isnan(v[0, 64:128]).all() and not np.isnan(v[0, :64]).any() and not np.isnan(v[0, 128:]).any()


def operand(rows, K, seed, lead=()):
    """Random codes and scales that vary by block: (device codes, device slabs, 64-bit values)."""
    r = np.random.default_rng(seed)
    codes = r.integers(0, 256, (*lead, rows, K // 2), dtype=np.uint8)
    rows_ = r.integers(117, 128, (*lead, rows, K // 32)).astype(np.uint8)
    return torch.from_numpy(codes).cuda(), torch.from_numpy(mx4.slabs(rows_)).cuda(), mx4.values(codes, rows_)


# every kernel: few rows, tiles of 64, 128 and 256 rows; K of part of a step, one
# step, a ragged number; N below and above a tile, odd
SHAPES = [(1, 32, 1), (1, 3840, 96), (5, 288, 33), (16, 256, 16), (17, 512, 40), (33, 1056, 257), (64, 96, 300),
          (65, 512, 256), (100, 800, 129), (128, 3840, 260), (129, 256, 512), (300, 1312, 513), (512, 64, 24),
          (513, 512, 256), (700, 1056, 1000), (1030, 288, 77), (2100, 96, 2560), (2100, 32, 2561), (3900, 288, 2300),
          (3900, 96, 2303), (20, 1824, 8200), (50, 1824, 8259)]


@pytest.mark.parametrize("M,K,N", SHAPES)
@pytest.mark.parametrize("out", ["f32", "bf16", "f16"])
def test_gemm(M, K, N, out):
    need_gpu()
    a, sa, av = operand(M, K, M + N)
    w, sw, wv = operand(N, K, M + N + 1)
    ref, bound = av @ wv.T, mx4.product_bound(av, wv)
    got = w4.w4a4_gemm_mx4(a, sa, w, sw, out_dtype=DT[out])
    assert got.shape == (M, N)
    mx4.close(as64(got), ref, bound, out)
    b = torch.randn(N, device="cuda").to(DT[out])
    got = w4.w4a4_gemm_mx4(a, sa, w, sw, bias=b, out_dtype=DT[out])
    mx4.close(as64(got), ref + as64(b), bound + 2.0 ** -24 * (np.abs(ref) + np.abs(as64(b))), out)


def test_gemm_plans_cover_the_shapes():
    names = {w4.w4a4_gemm_mx4_plan(M, K, N) for M, K, N in SHAPES}
    assert names == {"skinny", "tile64", "tile128", "tile256"}
    # 16-bit outputs whose rows a tile's 31-bit offsets do not reach across
    assert w4.w4a4_gemm_mx4_plan(1000, 64, 1 << 22) == "skinny" != w4.w4a4_gemm_mx4_plan(1000, 64, (1 << 22) - 256)


def test_gemm_nan_scales_reach_their_outputs_only():
    need_gpu()
    for M, N in ((4, 40), (90, 300), (300, 300), (600, 300)):
        a, sa, av = operand(M, 512, 3)
        w, sw, wv = operand(N, 512, 4)
        sa[1, M - 1, 2] = 255
        sw[0, 7, 5] = 255
        av[M - 1, 320:352] = np.nan                          # block 10
        wv[7, 160:192] = np.nan
        got = as64(w4.w4a4_gemm_mx4(a, sa, w, sw, out_dtype=torch.float32))
        nan = np.zeros((M, N), bool)
        nan[M - 1, :] = True
        nan[:, 7] = True
        assert np.array_equal(np.isnan(got), nan)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M", [1, 40, 200, 600])
def test_linear_is_quantizer_and_product(M, dtype):
    need_gpu()
    K, N, g = 768, 321, 128
    si, sid = signs(g, 1)
    h = w4.Hadamard(g, sid)
    x = draw_x(M, K, dtype, 8)
    w, sw, wv = operand(N, K, 9)
    b = torch.randn(N, device="cuda").to(DT[dtype])
    got = w4.w4a4_linear_mx4(x, w, sw, h=h, bias=b)
    codes, scales = w4.w4a4_quantize_mx4(x, h)
    assert torch.equal(got, w4.w4a4_gemm_mx4(codes, scales, w, sw, bias=b, out_dtype=DT[dtype]))
    rc, rs = mx4.quantize(mx4.rotate(x.cpu().float().numpy(), g, si, None))
    av = mx4.values(rc, rs)
    ref = av @ wv.T
    mx4.close(as64(got), ref + as64(b), mx4.product_bound(av, wv) + 2.0 ** -24 * (np.abs(ref) + np.abs(as64(b))), dtype)
    # leading dimensions, caller's output and workspace
    ws = torch.empty(w4.w4a4_linear_mx4_workspace_size(M, K), dtype=torch.uint8, device="cuda")
    out = torch.empty((M, N), dtype=DT[dtype], device="cuda")
    same = w4.w4a4_linear_mx4(x.view(1, M, K), w, sw, h=h, bias=b, workspace=ws, out=out)
    assert same.shape == (1, M, N) and torch.equal(out, got)


def test_empty_and_other_streams():
    need_gpu()
    w, sw, wv = operand(64, 256, 1)
    x = draw_x(0, 256, "bf16", 1)
    assert w4.w4a4_linear_mx4(x, w, sw).shape == (0, 64)
    codes, scales = w4.w4a4_quantize_mx4(x)
    assert codes.shape == (0, 128) and scales.shape == (1, 0, 8)
    assert w4.w4a4_dequantize_mx4(codes, scales).shape == (0, 256)
    x = draw_x(300, 256, "bf16", 2)
    ref = w4.w4a4_linear_mx4(x, w, sw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = w4.w4a4_linear_mx4(x, w, sw)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, ref)


def test_graph_replays():
    need_gpu()
    w, sw, _ = operand(256, 512, 1)
    x = draw_x(300, 512, "bf16", 2)
    out = torch.empty((300, 256), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(w4.w4a4_linear_mx4_workspace_size(300, 512), dtype=torch.uint8, device="cuda")
    w4.w4a4_linear_mx4(x, w, sw, workspace=ws, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w4.w4a4_linear_mx4(x, w, sw, workspace=ws, out=out)
    for seed in range(4):
        x.copy_(draw_x(300, 512, "bf16", 20 + seed))
        ref = w4.w4a4_linear_mx4(x, w, sw)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)


def test_offsets_past_32_bits():
    """An activation of more than 2^32 bytes, an output of more than 2^32 elements' bytes."""
    need_gpu()
    M, K, N = 600_001, 4096, 4096
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    rows = [0, 1, 524_287, 524_288, 524_289, 599_999, 600_000]
    tail = draw_x(len(rows), K, "bf16", 3)
    x[rows] = tail
    w, sw, _ = operand(N, K, 4)
    codes, scales = w4.w4a4_quantize_mx4(x)
    rc, rs = w4.w4a4_quantize_mx4(tail)
    assert torch.equal(codes[rows], rc) and torch.equal(scales[:, rows], rs)
    out = w4.w4a4_gemm_mx4(codes, scales, w, sw)
    small = w4.w4a4_gemm_mx4(rc, rs, w, sw, out_dtype=torch.float32)
    assert torch.allclose(out[rows].float(), small, rtol=2.0 ** -8, atol=1e-6 * small.abs().max().item())
    assert bool((out[2:524_287] == 0).all()) and bool((out[524_290:599_999] == 0).all())
    back = w4.w4a4_dequantize_mx4(codes, scales)
    assert torch.equal(back[rows], w4.w4a4_dequantize_mx4(rc, rs))


def test_outputs_of_8_mb_a_row():
    """More columns than a tile's offsets reach across: every 4096 of them the same weights.
    One block of k, so the sums are exact in any order."""
    need_gpu()
    M, K, N, times = 300, 32, 4096, 1024
    a, sa, _ = operand(M, K, 1)
    w, sw, _ = operand(N, K, 2)
    assert w4.w4a4_gemm_mx4_plan(M, K, N * times) == "skinny" != w4.w4a4_gemm_mx4_plan(M, K, N)
    out = w4.w4a4_gemm_mx4(a, sa, w.repeat(times, 1), sw.repeat(1, times, 1))
    assert bool((out.view(M, times, N) == w4.w4a4_gemm_mx4(a, sa, w, sw)[:, None]).all())

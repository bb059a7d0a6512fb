"""GPU tests of the block-scaled fp8 quantisers, their inverses and the dense product,
against plain forms in 64 bits (tests/fp8.py)."""
import numpy as np
import pytest
import torch

from tests import fp8, mx4
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def seeded():
    torch.manual_seed(7)

import bit_quantized_linear_rotate_amd as w4  # noqa: E402

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
F8 = torch.float8_e4m3fn


def as64(t):
    return t.detach().double().cpu().numpy()


def raw(codes):
    return codes.view(torch.uint8).cpu().numpy()


def draw_x(M, K, dtype, seed=0, scale=1.0):
    r = np.random.default_rng(seed)
    x = r.standard_normal((M, K)) * scale * np.where(r.random(K) < 0.02, 20.0, 1.0)
    return torch.from_numpy(x).to(DT[dtype]).cuda()


def signs(g, seed):
    r = np.random.default_rng(seed)
    return [torch.from_numpy((r.integers(0, 2, g) * 2 - 1).astype(np.int8)).cuda() for _ in range(2)]


def rows_operand(M, K, seed):
    """(codes, scales, 64-bit values) of random rows."""
    codes, s = fp8.quantize(np.random.default_rng(seed).standard_normal((M, K)))
    s = s.astype(np.float32)
    return (torch.from_numpy(codes).cuda().view(F8), torch.from_numpy(np.ascontiguousarray(s.T)).cuda(),
            fp8.values(codes, s))


def weights_operand(N, K, seed, E=0):
    r = np.random.default_rng(seed)
    got = [fp8.quantize(r.standard_normal((N, K)) * K ** -0.5 * r.uniform(0.5, 2), 128) for _ in range(E or 1)]
    codes, s = np.stack([g[0] for g in got]), np.stack([g[1] for g in got]).astype(np.float32)
    v = fp8.values(codes, s, 128)
    if not E:
        codes, s, v = codes[0], s[0], v[0]
    return torch.from_numpy(codes).cuda().view(F8), torch.from_numpy(s).cuda(), v


SIZES = [(1, 16), (1, 128), (3, 144), (17, 272), (40, 3840), (33, 1040), (129, 256)]


def check_codes(y, rows, codes, scales, exact):
    """y (64 bits, of fp32 values), scales (blocks, blocks).  exact: codes to the bit
    (16-bit values: the ratio's numerator has at most 14 bits, a border between codes 5,
    the divisor 11, so a ratio off a border is off by 2^-19 at least); else a ratio
    within 2^-22 of a border (its two roundings) may go either way."""
    want, s = fp8.quantize(y, rows)
    assert np.array_equal(np.isnan(scales), np.isnan(s))
    ok = ~np.isnan(s)
    assert (np.abs(scales[ok] - s[ok]) <= 2.0 ** -24 * s[ok]).all()
    if exact:
        assert np.array_equal(codes, want)
        return
    _, top = fp8.tops(y, rows)
    top = np.maximum(top, fp8.LEAST)
    v = np.abs(y) * 448 / top
    lo, hi = fp8.nearest_code(v * (1 - 2.0 ** -22)), fp8.nearest_code(v * (1 + 2.0 ** -22))
    assert ((codes & 127) >= lo).all() and ((codes & 127) <= hi).all()
    assert np.array_equal(codes >> 7, np.signbit(y))


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("M,K", SIZES)
def test_quantize_rows(M, K, dtype):
    need_gpu()
    x = draw_x(M, K, dtype, M + K)
    codes, scales = w4.w8a8_quantize_fp8(x)
    assert codes.dtype == F8 and scales.shape == (fp8.blocks(K), M)
    check_codes(as64(x), 1, raw(codes), as64(scales).T, dtype != "f32")
    v = fp8.values(raw(codes), as64(scales).T)
    for out in DT:
        mx4.close(as64(w4.w8a8_dequantize_fp8(codes, scales, DT[out])), v, 2.0 ** -24 * np.abs(v), out)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("N,K", SIZES + [(128, 128), (300, 512), (257, 400)])
def test_quantize_weights(N, K, dtype):
    need_gpu()
    w = draw_x(N, K, dtype, N)
    codes, scales = w4.w8a8_quantize_weights_fp8(w)
    check_codes(as64(w), 128, raw(codes), as64(scales), dtype != "f32")
    v = fp8.values(raw(codes), as64(scales), 128)
    for out in DT:
        mx4.close(as64(w4.w8a8_dequantize_weights_fp8(codes, scales, DT[out])), v, 2.0 ** -24 * np.abs(v), out)
    # several matrices: each as by itself, also from a strided view
    wide = torch.stack([w, w * 3, -w]).repeat(1, 1, 2)
    for view in (wide[:, :, :K].contiguous(), wide[:, :, :K], wide[:, :, :K].transpose(0, 1).contiguous().transpose(0, 1)):
        c3, s3 = w4.w8a8_quantize_weights_fp8(view)
        for e in range(3):
            ce, se = w4.w8a8_quantize_weights_fp8(view[e].contiguous())
            assert torch.equal(c3[e].view(torch.uint8), ce.view(torch.uint8)) and torch.equal(s3[e], se)
        assert torch.equal(w4.w8a8_dequantize_weights_fp8(c3, s3)[2], w4.w8a8_dequantize_weights_fp8(c3[2], s3[2]))


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("g", [16, 32, 64, 128, 256])
def test_quantize_rotated(g, dtype):
    need_gpu()
    M, K = 21, 768
    x = draw_x(M, K, dtype, g)
    si, so = signs(g, g)
    for h in (w4.Hadamard(g, si, so), w4.Hadamard(g), w4.Hadamard(g, sign_out=so)):
        # the rotation in fp32 with its order of butterflies is the definition
        y = mx4.rotate(as64(x), g, *(None if s is None else s.cpu().numpy() for s in (h.sign_in, h.sign_out)))
        codes, scales = w4.w8a8_quantize_fp8(x, h)
        check_codes(y.astype(np.float64), 1, raw(codes), as64(scales).T, False)
        codes, scales = w4.w8a8_quantize_weights_fp8(x, h)
        check_codes(y.astype(np.float64), 128, raw(codes), as64(scales), False)


@pytest.mark.parametrize("dtype", DT)
def test_quantize_strided(dtype):
    need_gpu()
    x = draw_x(70, 416, dtype, 3)
    want = w4.w8a8_quantize_fp8(x.contiguous())
    wide = draw_x(70, 500, dtype, 3)
    wide[:, 1:417] = x
    steps = torch.zeros(70, 832, dtype=DT[dtype], device="cuda")
    steps[:, ::2] = x
    for v in (x.t().contiguous().t(), wide[:, 1:417], steps[:, ::2], x.view(7, 10, 416)):
        got = w4.w8a8_quantize_fp8(v)
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want))


def test_quantize_extremes():
    """Zeros, the smallest and largest values, infinities and NaN, each in its own block."""
    need_gpu()
    big = float(torch.finfo(torch.float32).max)
    x = torch.randn(9, 384, device="cuda")
    x[0] = 0
    x[1] = 2.0 ** -149
    x[2, :128] = 2.0 ** -126
    x[3] *= big / 8
    x[4, 5] = big
    x[5, 130] = float("inf")
    x[6, 300] = float("nan")
    x[7, 0] = -float("inf")
    x[8] *= 2.0 ** -120
    codes, scales = w4.w8a8_quantize_fp8(x)
    y, s = as64(x), as64(scales).T
    fine = np.isfinite(fp8.tops(np.where(np.isfinite(y), y, np.inf), 1)[1])
    assert np.array_equal(np.isnan(np.repeat(s, 128, 1)), ~fine) and (raw(codes)[~fine] == 0).all()
    y0 = np.where(fine, y, 0.0)
    want = np.where(np.isnan(s), fp8.LEAST / 448, s)
    check_codes(y0, 1, np.where(fine, raw(codes), np.signbit(y0) << 7).astype(np.uint8), want, False)
    assert np.isnan(as64(w4.w8a8_dequantize_fp8(codes, scales))[~fine]).all()
    wc, ws = w4.w8a8_quantize_weights_fp8(x)
    assert bool(torch.isnan(ws).all()) and int(raw(wc).max()) == 0   # every block of three holds one
    wc, ws = w4.w8a8_quantize_weights_fp8(x[:4])
    check_codes(as64(x[:4]), 128, raw(wc), as64(ws), False)


def test_ties_go_to_the_even_code():
    need_gpu()
    mid = (fp8.GRID[1:] + fp8.GRID[:-1]) / 2
    y = np.zeros((4, 128))
    y[:, 0] = 448
    for i, part in enumerate(np.array_split(np.concatenate([mid, -mid[:126]]), 4)):
        y[i, 1:1 + len(part)] = part
    for p in (0, -3, 40, -60):
        codes, scales = w4.w8a8_quantize_fp8(torch.from_numpy(y * 2.0 ** p).float().cuda())
        check_codes(y * 2.0 ** p, 1, raw(codes), as64(scales).T, True)


# rows, K, N: every kernel, widths that no tile divides, K that ends inside a block
GEMMS = [(1, 16, 16), (1, 3840, 48), (5, 272, 130), (16, 400, 257), (17, 128, 64), (40, 1040, 300), (64, 512, 1000),
         (100, 640, 256), (129, 272, 513), (200, 1296, 2304), (333, 384, 1001), (700, 528, 2305), (1500, 272, 3841),
         (2049, 1040, 2560), (4100, 272, 1280), (3000, 400, 4099), (5000, 144, 2305)]


def test_sizes_reach_every_kernel():
    assert {w4.w8a8_gemm_fp8_plan(M, K, N) for M, K, N in GEMMS} == {"skinny", "tile64", "tile128", "tile256"}


@pytest.mark.parametrize("M,K,N", GEMMS)
def test_gemm(M, K, N):
    need_gpu()
    a, sa, av = rows_operand(M, K, M)
    w, sw, wv = weights_operand(N, K, N)
    ref = av @ wv.T
    for out in DT:
        bound = fp8.product_bound(av, wv, out)
        mx4.close(as64(w4.w8a8_gemm_fp8(a, sa, w, sw, out_dtype=DT[out])), ref, bound, out)
        b = torch.randn(N, device="cuda").to(DT[out])
        bv = as64(b)
        got = w4.w8a8_gemm_fp8(a, sa, w, sw, bias=b, out_dtype=DT[out])
        mx4.close(as64(got), ref + bv, bound + 2.0 ** -24 * (np.abs(ref) + np.abs(bv)), out)


@pytest.mark.parametrize("M,K,N", GEMMS)
def test_gemm_of_small_integers_is_exact(M, K, N):
    """Codes of integers up to 4 under powers of two: every sum is exact (products up to
    16, blocks up to 2^11, scales' products 2^-2 .. 2^2, sums below 2^24 quarters), so
    the outputs are the exact ones rounded."""
    need_gpu()
    r = np.random.default_rng(M + N)
    a, w = r.integers(-4, 5, (M, K)).astype(np.float64), r.integers(-4, 5, (N, K)).astype(np.float64)
    sa = 2.0 ** r.integers(-1, 2, (M, fp8.blocks(K)))
    sw = 2.0 ** r.integers(-1, 2, (fp8.blocks(N), fp8.blocks(K)))
    full = lambda v, s, rows: v * np.repeat(np.repeat(s, rows, 0)[:v.shape[0]], 128, 1)[:, :K]  # noqa: E731
    ref = full(a, sa, 1) @ full(w, sw, 128).T
    put = lambda v: torch.from_numpy(v).float().to(F8).cuda()  # noqa: E731
    sat, swt = torch.from_numpy(np.ascontiguousarray(sa.T)).float().cuda(), torch.from_numpy(sw).float().cuda()
    for out in DT:
        got = w4.w8a8_gemm_fp8(put(a), sat, put(w), swt, out_dtype=DT[out])
        assert torch.equal(got.cpu(), torch.from_numpy(ref).to(DT[out]))


def test_gemm_is_the_same_every_time():
    need_gpu()
    for M, K, N in ((3, 1040, 300), (700, 528, 2305)):
        a, sa, _ = rows_operand(M, K, 1)
        w, sw, _ = weights_operand(N, K, 2)
        first = w4.w8a8_gemm_fp8(a, sa, w, sw)
        for _ in range(3):
            assert torch.equal(first, w4.w8a8_gemm_fp8(a, sa, w, sw))


def test_gemm_nan_and_extreme_scales():
    need_gpu()
    for M in (4, 300):
        a, sa, av = rows_operand(M, 400, 1)
        w, sw, wv = weights_operand(300, 400, 2)
        sa, sw = sa.clone(), sw.clone()
        sa[1, 2] = float("nan")      # a row's block
        sw[2, 3] = float("nan")      # columns 256 .. 299
        got = as64(w4.w8a8_gemm_fp8(a, sa, w, sw, out_dtype=torch.float32))
        bad = np.zeros((M, 300), bool)
        bad[2] = bad[:, 256:] = True
        assert np.array_equal(np.isnan(got), bad)
        ref, bound = av @ wv.T, fp8.product_bound(av, wv, "f32")
        mx4.close(got[~bad], ref[~bad], bound[~bad], "f32")
        # 2^-60 times 2^60
        a, sa, av = rows_operand(M, 400, 1)
        w, sw, wv = weights_operand(300, 400, 2)
        mx4.close(as64(w4.w8a8_gemm_fp8(a, sa * 2.0 ** -60, w, sw * 2.0 ** 60, out_dtype=torch.float32)), ref, bound, "f32")


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("M,g", [(1, 64), (30, 0), (300, 128)])
def test_linear(M, g, dtype):
    need_gpu()
    K, N = 640, 272
    x = draw_x(M, K, dtype, 5).view(1, M, K)
    h = w4.Hadamard(g, *signs(g, 1)) if g else None
    w, sw = w4.w8a8_quantize_weights_fp8(torch.randn(N, K, device="cuda"), h)
    b = torch.randn(N, device="cuda").to(DT[dtype])
    codes, scales = w4.w8a8_quantize_fp8(x, h)
    want = w4.w8a8_gemm_fp8(codes, scales, w, sw, bias=b, out_dtype=DT[dtype])
    got = w4.w8a8_linear_fp8(x, w, sw, h=h, bias=b)
    assert got.shape == (1, M, N) and torch.equal(got[0], want)
    out = torch.empty(M, N, dtype=torch.float32, device="cuda")
    ws = torch.empty(w4.w8a8_linear_fp8_workspace_size(M, K), dtype=torch.uint8, device="cuda")
    got = w4.w8a8_linear_fp8(x[0], w, sw, h=h, bias=b, workspace=ws, out=out)
    assert got.data_ptr() == out.data_ptr()
    assert torch.equal(got, w4.w8a8_gemm_fp8(codes, scales, w, sw, bias=b, out_dtype=torch.float32))


def test_empty_and_narrow():
    need_gpu()
    w, sw, _ = weights_operand(64, 256, 1)
    x = torch.zeros(0, 256, device="cuda", dtype=torch.bfloat16)
    assert w4.w8a8_linear_fp8(x, w, sw).shape == (0, 64)
    c, s = w4.w8a8_quantize_fp8(x)
    assert c.shape == (0, 256) and s.shape == (2, 0) and w4.w8a8_dequantize_fp8(c, s).shape == (0, 256)
    c, s = w4.w8a8_quantize_weights_fp8(x)
    assert c.shape == (0, 256) and s.shape == (0, 2)
    assert w4.w8a8_linear_fp8(torch.ones(3, 256, device="cuda"), w[:0], sw[:0]).shape == (3, 0)


def test_streams_and_graph_replays():
    """On a side stream, and captured: replays read new inputs and leave the eager result."""
    need_gpu()
    K, N = 1040, 512
    w, sw = w4.w8a8_quantize_weights_fp8(torch.randn(N, K, device="cuda"))
    for M in (2, 400):
        x = draw_x(M, K, "bf16", M)
        want = w4.w8a8_linear_fp8(x, w, sw)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = w4.w8a8_linear_fp8(x, w, sw)
        side.synchronize()
        assert torch.equal(got, want)
        ws = torch.empty(w4.w8a8_linear_fp8_workspace_size(M, K), dtype=torch.uint8, device="cuda")
        held = x.clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = w4.w8a8_linear_fp8(held, w, sw, workspace=ws)
        for i in range(4):
            held.copy_(x * (i + 1))
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, w4.w8a8_linear_fp8(held, w, sw))

"""GPU tests of the products grouped by expert, routing, combining and the expert
layer, against plain forms in 64 bits (tests/mx4.py)."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from tests import mx4
from tests.gpu_util import need_gpu
from tests.test_gpu_mx4 import DT, as64, draw_x, operand, signs

pytestmark = pytest.mark.gpu

import bit_quantized_linear_rotate_amd as w4  # noqa: E402


def offsets_of(counts):
    return torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)).cuda()


# counts per expert (empty ones, one row, tiles and tiles plus one), rows past the last
CASES = {
    "skinny one": ([1], 0),
    "skinny": ([0, 3, 1, 0, 16, 17, 2, 0], 5),
    "skinny two": ([33, 0, 20, 64, 5, 31], 0),
    "tile64": ([64, 65, 0, 200, 1, 128, 90], 3),
    "tile128": ([128, 129, 0, 600, 255, 1], 9),
    "tile256": ([256, 2049, 0, 513, 1, 700], 1),
    "large": ([700, 1, 900, 333, 0, 513, 64], 5),
    "larger": ([2300, 0, 1, 2049, 513], 2),
    "largest": ([2600, 1, 2049, 513], 2),
    "many experts": ([i % 3 for i in range(200)], 0),
    "nothing routed": ([0, 0, 0], 7),
}


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("K,N", [(512, 256), (288, 77), (288, 2304), (96, 2561), (1056, 2304)])
def test_grouped_gemm(name, K, N):
    need_gpu()
    counts, extra = CASES[name]
    E, R = len(counts), sum(counts) + extra
    r = np.random.default_rng(R)
    T = max(1, R // 2)
    a, sa, av = operand(T, K, 1)
    w, sw, wv = operand(N, K, 2, (E,))
    rows = r.integers(0, T, R).astype(np.int32)
    off = offsets_of(counts)
    o = off.cpu().numpy()
    ref, bound = np.zeros((R, N)), np.zeros((R, N))
    b = torch.randn(E, N, device="cuda").to(torch.bfloat16)
    for e in range(E):
        at = slice(o[e], o[e + 1])
        x = av[rows[at]]
        ref[at] = x @ wv[e].T + as64(b[e])
        bound[at] = mx4.product_bound(x, wv[e]) + 2.0 ** -24 * (np.abs(ref[at]) + 2 * np.abs(as64(b[e])))
    rt = torch.from_numpy(rows).cuda()
    for out in DT:
        got = w4.w4a4_grouped_gemm_mx4(a, sa, w, sw, off, rows=rt, bias=b, out_dtype=DT[out])
        mx4.close(as64(got), ref, bound, out)
        assert bool((got[o[E]:] == 0).all())
    # without a row index: the rows laid out already
    if R > 0:
        ga, gsa = a[rt.long()].contiguous(), sa[:, rt.long()].contiguous()
        assert torch.equal(w4.w4a4_grouped_gemm_mx4(ga, gsa, w, sw, off, bias=b), w4.w4a4_grouped_gemm_mx4(
            a, sa, w, sw, off, rows=rt, bias=b))


def test_grouped_rows_outside_the_codes_are_zero_rows():
    need_gpu()
    for counts in ([9, 4], [100, 80], [700, 400]):
        R, T, K, N = sum(counts), 50, 256, 96
        a, sa, av = operand(T, K, 1)
        w, sw, wv = operand(N, K, 2, (2,))
        rows = np.random.default_rng(1).integers(0, T, R).astype(np.int32)
        rows[3], rows[R - 1], rows[5] = -1, T, 2 ** 31 - 1
        got = as64(w4.w4a4_grouped_gemm_mx4(a, sa, w, sw, offsets_of(counts), rows=torch.from_numpy(rows).cuda(),
                                            out_dtype=torch.float32))
        assert (got[[3, 5, R - 1]] == 0).all()
        x = np.where(((rows >= 0) & (rows < T))[:, None], av[np.clip(rows, 0, T - 1)], 0)
        for e, at in enumerate((slice(0, counts[0]), slice(counts[0], R))):
            mx4.close(got[at], x[at] @ wv[e].T, mx4.product_bound(x[at], wv[e]), "f32")


def check_gated(codes, scales, g, u, eg, eu):
    """MX4 form of silu(g) u against 64 bits: a code may be the neighbour's only where the
    fp32 error of the value reaches the boundary between them, a scale only where the
    error of the block's largest value reaches a power of two."""
    v = mx4.silu(g) * u
    # |silu'| <= 1.1; exp, division and products: a few units of fp32
    err = 1.1 * np.abs(u) * eg + np.abs(mx4.silu(g)) * eu + 1.1 * eg * eu + 2.0 ** -20 * np.abs(v) + 2.0 ** -126
    R, F = v.shape
    got = mx4.values(codes, scales)
    lo, hi = np.abs(v) - err, np.abs(v) + err
    b = lambda t: t.reshape(R, F // 32, 32)  # noqa: E731
    X = scales.astype(np.int64) - 127
    assert (X >= mx4.scale_exponent(np.maximum(b(lo).max(-1), 0))).all() and (X <= mx4.scale_exponent(b(hi).max(-1))).all()
    s = np.exp2(X.astype(np.float64))[..., None]
    least = mx4.GRID[mx4.nearest_code(np.maximum(b(lo), 0) / s)]
    most = mx4.GRID[mx4.nearest_code(b(hi) / s)]
    m = np.abs(b(got)) / s
    assert ((m >= least) & (m <= most)).all()
    sure = (np.abs(v) > err) & (got != 0)
    assert (np.signbit(got) == np.signbit(v))[sure].all()


def test_cases_reach_every_kernel():
    shapes = {False: ((512, 256), (288, 77), (288, 2304), (96, 2561), (1056, 2304)),
              True: ((512, 512), (288, 192), (256, 320), (288, 2368), (1056, 2368))}
    for gated, widths in shapes.items():
        got = {w4.w4a4_gemm_mx4_plan(sum(c) + x, k, n, len(c), gated) for c, x in CASES.values() for k, n in widths}
        assert got == {"skinny", "tile64", "tile128", "tile256"}, (gated, got)


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("K,F", [(512, 256), (288, 96), (256, 160), (288, 1184), (1056, 1184)])
def test_grouped_gated(name, K, F):
    need_gpu()
    counts, extra = CASES[name]
    E, R = len(counts), sum(counts) + extra
    T = max(1, R // 2)
    a, sa, av = operand(T, K, 1)
    w, sw, wv = operand(2 * F, K, 2, (E,))
    sa = (sa.int() - 5).clamp(min=0).to(torch.uint8)      # values of the size activations have
    av = av * 2.0 ** -5
    rows = np.random.default_rng(R).integers(0, T, R).astype(np.int32)
    off = offsets_of(counts)
    o = off.cpu().numpy()
    b = (torch.randn(E, 2 * F, device="cuda") * 0.5).to(torch.bfloat16)
    codes, scales = w4.w4a4_grouped_gated_mx4(a, sa, w, sw, off, rows=torch.from_numpy(rows).cuda(), bias=b)
    codes, full = codes.cpu().numpy(), scales.cpu().numpy()
    srows = mx4.unslab(full, F)
    assert np.array_equal(full, mx4.slabs(srows))          # the unused bytes are zero
    assert not codes[o[E]:].any() and not srows[o[E]:].any()
    for e in range(E):
        at = slice(o[e], o[e + 1])
        if o[e] == o[e + 1]:
            continue
        x = av[rows[at]]
        y, bound = x @ wv[e].T + as64(b[e]), mx4.product_bound(x, wv[e])
        bound = bound + 2.0 ** -24 * (np.abs(y) + 2 * np.abs(as64(b[e])))
        check_gated(codes[at], srows[at], y[:, :F], y[:, F:], bound[:, :F], bound[:, F:])


def logits_of(T, E, dtype, seed):
    r = np.random.default_rng(seed)
    l = np.round(r.standard_normal((T, E)) * 3, 1)         # ties
    l[::5] = np.where(r.random((len(l[::5]), E)) < 0.7, -np.inf, l[::5])
    l[3::17] = -np.inf
    l[4::13, 0] = np.nan
    l[6::19] = np.where(r.random((len(l[6::19]), E)) < 0.5, 0.0, -0.0)
    return torch.from_numpy(l).to(DT[dtype]).cuda()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (5, 64, 8), (64, 32, 4), (65, 65, 3), (200, 128, 8), (130, 257, 5),
                                   (700, 16, 16), (70, 1024, 32), (9000, 40, 2)])
def test_route(T, E, k, dtype):
    need_gpu()
    l = logits_of(T, E, dtype, T + E)
    for renorm in (True, False):
        got = w4.w4a4_route_experts(l, k, renormalize=renorm)
        weights, experts, rows, pos, offsets = mx4.route(as64(l), k, renorm)
        for g, r in zip(got[1:], (experts, rows, pos, offsets)):
            assert g.dtype == torch.int32 and np.array_equal(g.cpu().numpy(), r)
        gw = as64(got[0])
        assert (np.abs(gw - weights) <= (E + 64) * 2.0 ** -24 * weights).all()


def test_route_strided_logits_and_no_tokens():
    need_gpu()
    wide = logits_of(100, 40, "f32", 1)
    a = w4.w4a4_route_experts(wide[:, 4:24], 3)
    b = w4.w4a4_route_experts(wide[:, 4:24].contiguous(), 3)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    got = w4.w4a4_route_experts(wide[:0], 3)
    assert got[0].shape == (0, 3) and bool((got[4] == 0).all()) and got[4].shape == (41,)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,k,N", [(1, 1, 1), (3, 4, 77), (70, 8, 256), (513, 3, 2056)])
def test_combine(T, k, N, dtype):
    need_gpu()
    r = np.random.default_rng(T)
    R = max(1, T * k - 2)
    y = torch.randn(R, N, device="cuda").to(DT[dtype])
    pos = r.integers(-1, R, (T, k)).astype(np.int32)
    pos[0] = -1                                            # a token with nothing
    w = torch.rand(T, k, device="cuda")
    got = w4.w4a4_combine_experts(y, torch.from_numpy(pos).cuda(), w)
    v = np.where((pos >= 0)[..., None], as64(y)[np.maximum(pos, 0)], 0) * as64(w)[..., None]
    mx4.close(as64(got), v.sum(1), (k + 1) * 2.0 ** -24 * np.abs(v).sum(1), dtype)


@pytest.mark.parametrize("T,E,k", [(1, 4, 2), (16, 32, 4), (300, 8, 2), (700, 6, 3), (64, 4, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_experts_is_its_parts(T, E, k, dtype):
    """The expert layer is the five calls, bit for bit; and it is the layer: within the
    quantisation noise of the hidden rows of the 64-bit layer on the same codes."""
    need_gpu()
    K, F, g = 512, 288, 64
    si, sid = signs(g, 3)
    h = w4.Hadamard(g, sid)
    x = draw_x(T, K, dtype, 1)
    l = logits_of(T, E, "f32", 2)
    w13, s13, v13 = operand(2 * F, K, 3, (E,))
    w2, s2, v2 = operand(K, F, 4, (E,))
    s13 = (s13.int() - 6).clamp(min=0).to(torch.uint8)
    got = w4.w4a4_experts_mx4(x, l, k, w13, s13, w2, s2, h=h)
    weights, experts, rows, pos, off = w4.w4a4_route_experts(l, k)
    c, s = w4.w4a4_quantize_mx4(x, h)
    ac, as_ = w4.w4a4_grouped_gated_mx4(c, s, w13, s13, off, rows=rows)
    y = w4.w4a4_grouped_gemm_mx4(ac, as_, w2, s2, off, out_dtype=DT[dtype])
    assert torch.equal(got, w4.w4a4_combine_experts(y, pos, weights))
    # tokens with no expert are zeros
    none = (experts < 0).all(1)
    assert bool((got[none] == 0).all())
    # the layer from the MX4 codes of the hidden rows, in 64 bits
    act = mx4.values(ac.cpu().numpy(), mx4.unslab(as_.cpu().numpy(), F))
    o, p, wt = off.cpu().numpy(), pos.cpu().numpy(), as64(weights)
    yy, bound = np.zeros((T * k, K)), np.zeros((T * k, K))
    rel, _ = mx4.HALF_ULP[dtype]
    for e in range(E):
        at = slice(o[e], o[e + 1])
        yy[at] = act[at] @ v2[e].T
        bound[at] = mx4.product_bound(act[at], v2[e]) + rel * np.abs(yy[at])
    ref = (np.where((p >= 0)[..., None], yy[np.maximum(p, 0)], 0) * wt[..., None]).sum(1)
    lim = (np.where((p >= 0)[..., None], bound[np.maximum(p, 0)], 0) * wt[..., None]).sum(1)
    mag = (np.where((p >= 0)[..., None], np.abs(yy)[np.maximum(p, 0)], 0) * wt[..., None]).sum(1)
    mx4.close(as64(got), ref, lim + (k + 1) * 2.0 ** -24 * mag, dtype)


def test_experts_workspace_output_and_empty():
    need_gpu()
    T, E, k, K, F = 40, 6, 2, 256, 64
    x = draw_x(T, K, "bf16", 1)
    l = logits_of(T, E, "bf16", 2)
    w13, s13, _ = operand(2 * F, K, 3, (E,))
    w2, s2, _ = operand(K, F, 4, (E,))
    ref = w4.w4a4_experts_mx4(x, l, k, w13, s13, w2, s2)
    need = w4.w4a4_experts_mx4_workspace_size(T, K, F, E, k, torch.bfloat16)
    ws = torch.full((need,), 0xAB, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(x)
    w4.w4a4_experts_mx4(x, l, k, w13, s13, w2, s2, workspace=ws, out=out)
    assert torch.equal(out, ref)
    assert w4.w4a4_experts_mx4(x[:0], l[:0], k, w13, s13, w2, s2).shape == (0, K)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = w4.w4a4_experts_mx4(x, l, k, w13, s13, w2, s2)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, ref)


def test_example_block():
    """The example's block against single precision.  A value rounded to e2m1 under a
    power-of-two scale is off by 0.1 to 0.13 of itself (rms), so a product of two rounded
    operands by up to 0.19, gated products and the second product, whose operands carry that
    too, by up to 0.33; the block is a sum of both kinds."""
    need_gpu()
    spec = importlib.util.spec_from_file_location("mx4_expert_block", os.path.join(
        os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mx4_expert_block.py"))
    block = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(block)
    assert 0.05 < block.main(tokens=200, K=512, F=256, E=8, top_k=2, repeat=2) < 0.33

"""GPU tests of the fp8 products grouped by expert, routing by scores and the fp8
expert layer, against plain forms in 64 bits (tests/fp8.py)."""
import numpy as np
import pytest
import torch

from tests import fp8, mx4
from tests.gpu_util import need_gpu
from tests.test_gpu_fp8 import DT, F8, as64, draw_x, raw, rows_operand, signs, weights_operand

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def seeded():
    torch.manual_seed(7)

import bit_quantized_linear_rotate_amd as w4  # noqa: E402


def offsets_of(counts, first=0):
    return torch.from_numpy(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32) + np.int32(first)).cuda()


# counts per expert (empty ones, one row, tiles and tiles plus one), rows past the last
CASES = {
    "skinny one": ([1], 0),
    "skinny": ([0, 3, 1, 0, 16, 17, 2, 0], 5),
    "skinny two": ([33, 0, 20, 64, 5, 31], 0),
    "tile64": ([64, 65, 0, 200, 1, 128, 90], 3),
    "tile128": ([128, 129, 0, 600, 255, 1], 9),
    "tile256": ([256, 2049, 0, 513, 1, 700], 1),
    "large": ([700, 1, 900, 333, 0, 513, 64], 5),
    "largest": ([2600, 1, 2049, 513], 2),
    # (a workgroup's tiles change between ones with rows in the lower half alone and full ones)
    "few and many": ([3, 64, 40, 0, 33, 1, 64, 17] * 8, 2),
    "many experts": ([i % 3 for i in range(90)], 0),
    "nothing routed": ([0, 0, 0], 7),
}
WIDTHS = [(512, 256), (272, 77), (400, 2304), (16, 130), (1040, 2561)]
GATED = [(512, 256), (272, 128), (400, 1152), (1040, 384)]


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("K,N", WIDTHS)
def test_grouped_gemm(name, K, N):
    need_gpu()
    counts, extra = CASES[name]
    E, R = len(counts), sum(counts) + extra
    r = np.random.default_rng(R)
    T = max(1, R // 2)
    a, sa, av = rows_operand(T, K, 1)
    w, sw, wv = weights_operand(N, K, 2, E)
    rows = r.integers(0, T, R).astype(np.int32)
    off = offsets_of(counts)
    o = off.cpu().numpy()
    ref, bounds = np.zeros((R, N)), {out: np.zeros((R, N)) for out in ("f32", "bf16")}
    b = torch.randn(E, N, device="cuda").to(torch.bfloat16)
    for e in range(E):
        at = slice(o[e], o[e + 1])
        x = av[rows[at]]
        ref[at] = x @ wv[e].T + as64(b[e])
        for out in bounds:
            bounds[out][at] = fp8.product_bound(x, wv[e], out) + 2.0 ** -24 * (np.abs(ref[at]) + 2 * np.abs(as64(b[e])))
    rt = torch.from_numpy(rows).cuda()
    for out in DT:
        got = w4.w8a8_grouped_gemm_fp8(a, sa, w, sw, off, rows=rt, bias=b, out_dtype=DT[out])
        mx4.close(as64(got), ref, bounds["f32" if out == "f32" else "bf16"], out)
        assert bool((got[o[E]:] == 0).all())
    # without a row index: the rows laid out already
    ga, gsa = a.view(torch.uint8)[rt.long()].view(F8), sa[:, rt.long()].contiguous()
    assert torch.equal(w4.w8a8_grouped_gemm_fp8(ga, gsa, w, sw, off, bias=b),
                       w4.w8a8_grouped_gemm_fp8(a, sa, w, sw, off, rows=rt, bias=b))


def test_cases_reach_every_kernel():
    # (gated products are fp16 ones, whose tiles have 64 or 128 rows)
    for gated, widths, kernels in ((False, WIDTHS, {"tile64", "tile128", "tile256"}),
                                   (True, [(k, 2 * f) for k, f in GATED], {"tile64", "tile128"})):
        got = {w4.w8a8_gemm_fp8_plan(sum(c) + x, k, n, len(c), gated) for c, x in CASES.values() for k, n in widths}
        assert got == kernels, (gated, got)


def test_grouped_rows_outside_the_codes_are_zero_rows():
    need_gpu()
    for counts in ([9, 4], [100, 80], [700, 400]):
        R, T, K, N = sum(counts), 50, 272, 96
        a, sa, av = rows_operand(T, K, 1)
        w, sw, wv = weights_operand(N, K, 2, 2)
        rows = np.random.default_rng(1).integers(0, T, R).astype(np.int32)
        rows[3], rows[R - 1], rows[5] = -1, T, 2 ** 31 - 1
        got = as64(w4.w8a8_grouped_gemm_fp8(a, sa, w, sw, offsets_of(counts), rows=torch.from_numpy(rows).cuda(),
                                            out_dtype=torch.float32))
        assert (got[[3, 5, R - 1]] == 0).all()
        x = np.where(((rows >= 0) & (rows < T))[:, None], av[np.clip(rows, 0, T - 1)], 0)
        for e, at in enumerate((slice(0, counts[0]), slice(counts[0], R))):
            mx4.close(got[at], x[at] @ wv[e].T, fp8.product_bound(x[at], wv[e], "f32"), "f32")


def test_rows_before_the_first_offset_are_zeros():
    need_gpu()
    for counts in ([3, 4], [300, 1, 500]):
        first, K, E = 11, 272, len(counts)
        R = first + sum(counts) + 5
        a, sa, _ = rows_operand(R, K, 1)
        w, sw, _ = weights_operand(256, K, 2, E)
        got = w4.w8a8_grouped_gemm_fp8(a, sa, w, sw, offsets_of(counts, first))
        assert bool((got[:first] == 0).all()) and bool((got[-5:] == 0).all())
        inner = slice(first, R - 5)
        a2, sa2 = a.view(torch.uint8)[inner].contiguous().view(F8), sa[:, inner].contiguous()
        assert torch.equal(got[inner], w4.w8a8_grouped_gemm_fp8(a2, sa2, w, sw, offsets_of(counts)))
        codes, scales = w4.w8a8_grouped_gated_fp8(a, sa, w, sw, offsets_of(counts, first))
        c2, s2 = w4.w8a8_grouped_gated_fp8(a2, sa2, w, sw, offsets_of(counts))
        assert (raw(codes)[:first] == 0).all() and (raw(codes)[-5:] == 0).all()
        assert bool((scales[:, :first] == 0).all()) and bool((scales[:, -5:] == 0).all())
        assert np.array_equal(raw(codes)[inner], raw(c2)) and torch.equal(scales[:, inner], s2)


@pytest.mark.parametrize("name", CASES)
@pytest.mark.parametrize("K,F", GATED)
def test_grouped_gated(name, K, F):
    need_gpu()
    counts, extra = CASES[name]
    E, R = len(counts), sum(counts) + extra
    T = max(1, R // 2)
    a, sa, av = rows_operand(T, K, 3)
    w, sw, wv = weights_operand(2 * F, K, 4, E)
    rows = np.random.default_rng(R).integers(0, T, R).astype(np.int32)
    off, rt = offsets_of(counts), torch.from_numpy(rows).cuda()
    o = off.cpu().numpy()
    for bias in (None, torch.randn(E, 2 * F, device="cuda").to(torch.float16)):
        codes, scales = w4.w8a8_grouped_gated_fp8(a, sa, w, sw, off, rows=rt, bias=bias)
        assert codes.shape == (R, F) and scales.shape == (F // 128, R)
        c, s = raw(codes), as64(scales).T
        for e in range(E):
            at = slice(o[e], o[e + 1])
            x = av[rows[at]]
            y, err = x @ wv[e].T, fp8.product_bound(x, wv[e], "f32")
            if bias is not None:
                y = y + as64(bias[e])
                err = err + 2.0 ** -24 * (np.abs(y) + 2 * np.abs(as64(bias[e])))
            fp8.check_gated(c[at], s[at], y[:, :F], y[:, F:], err[:, :F], err[:, F:])
        assert (c[o[E]:] == 0).all() and (s[o[E]:] == 0).all()


def test_gated_extremes():
    """Gates far below and above zero, all-zero rows, a NaN."""
    need_gpu()
    for counts in ([5], [150]):
        R, K, F = counts[0], 128, 128
        a, sa, av = rows_operand(R, K, 1)
        w, sw, wv = weights_operand(2 * F, K, 2, 1)
        bias = torch.zeros(1, 2 * F, device="cuda")
        bias[0, :F] = -200.0       # silu vanishes: values below any code
        codes, scales = w4.w8a8_grouped_gated_fp8(a, sa, w, sw, offsets_of(counts), bias=bias)
        assert (raw(codes) & 127 == 0).all() and np.allclose(as64(scales), fp8.LEAST / 448, rtol=1e-6)
        bias[0, :F] = 200.0        # silu is the identity
        codes, scales = w4.w8a8_grouped_gated_fp8(a, sa, w, sw, offsets_of(counts), bias=bias)
        y, err = av @ wv[0].T, fp8.product_bound(av, wv[0], "f32")
        y[:, :F] += 200
        fp8.check_gated(raw(codes), as64(scales).T, y[:, :F], y[:, F:], err[:, :F] + 2.0 ** -15, err[:, F:])
        za = torch.zeros_like(a.view(torch.uint8)).view(F8)
        codes, scales = w4.w8a8_grouped_gated_fp8(za, sa, w, sw, offsets_of(counts))
        assert (raw(codes) & 127 == 0).all() and np.allclose(as64(scales), fp8.LEAST / 448, rtol=1e-6)
        sa = sa.clone()
        sa[0, 2] = float("nan")
        codes, scales = w4.w8a8_grouped_gated_fp8(a, sa, w, sw, offsets_of(counts))
        assert np.array_equal(np.isnan(as64(scales)[0]), np.arange(R) == 2) and (raw(codes)[2] == 0).all()


# ---- routing by scores --------------------------------------------------------

def logits_of(T, E, dtype, seed, masked=True):
    r = np.random.default_rng(seed)
    l = r.standard_normal((T, E)) + r.standard_normal(E)
    if masked:
        l[::7][r.random((len(l[::7]), E)) < 0.6] = -np.inf
        l[::13] = -np.inf
        l[5::17, 0] = np.nan
    return torch.from_numpy(l).to(DT[dtype]).cuda()


def check_route(l, k, **how):
    got = [as64(v) for v in w4.w4a4_route_experts_scored(l, k, **how)]
    plain = dict(how)
    if plain.get("bias") is not None:
        plain["bias"] = as64(plain["bias"])
    plain["scale"] = float(np.float32(plain.get("scale", 1.0)))
    want = fp8.route(as64(l), k, **plain)
    for g, w in zip(got[1:], want[1:]):
        assert np.array_equal(g, w)
    # one rounding to fp32, some of double precision (exp, sum, divisions: 2^-48 at most)
    assert (np.abs(got[0] - want[0]) <= (2.0 ** -24 + 2.0 ** -48) * np.abs(want[0]) + 2.0 ** -149).all()


ROUTES = [(1, 1, 1, 1, 1), (1, 4, 2, 1, 1), (3, 8, 8, 1, 1), (32, 32, 4, 4, 2), (65, 64, 6, 8, 3), (300, 128, 8, 1, 1),
          (40, 160, 6, 8, 3), (129, 256, 8, 8, 4), (70, 256, 16, 64, 17), (50, 256, 20, 4, 2), (33, 384, 8, 16, 5),
          (17, 1024, 32, 64, 9), (1500, 48, 3, 6, 2), (20, 12, 12, 12, 12), (30, 20, 3, 5, 3),
          # as many choices as lanes leave room for, one more, and all experts
          (40, 200, 14, 1, 1), (40, 200, 15, 1, 1), (20, 14, 14, 1, 1), (21, 16, 16, 4, 4)]


@pytest.mark.parametrize("T,E,k,groups,top_groups", ROUTES)
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_route(T, E, k, groups, top_groups, scores):
    need_gpu()
    bias = torch.from_numpy(0.2 * np.random.default_rng(E).standard_normal(E)).float().cuda()
    how = dict(scores=scores, groups=groups, top_groups=top_groups)
    for dtype in DT:
        l = logits_of(T, E, dtype, T + E)
        check_route(l, k, group_best=1, renormalize=True, **how)
        check_route(l, k, group_best=2, renormalize=False, scale=2.5, **how)
        check_route(l, k, group_best=2, renormalize=True, scale=2.5, bias=bias, **how)
        check_route(l, k, group_best=1, renormalize=False, bias=bias, **how)


def test_route_ties_go_to_the_lower_index():
    need_gpu()
    for E, k, groups, top in ((8, 3, 4, 2), (64, 5, 8, 3), (256, 8, 8, 4), (512, 8, 16, 4)):
        l = torch.zeros(70, E, device="cuda")
        l[1::2] = torch.randint(-1, 2, (35, E), generator=torch.Generator().manual_seed(E)).float().cuda()
        for best in (1, 2):
            for bias in (None, torch.zeros(E, device="cuda")):
                for scores in ("softmax", "sigmoid"):
                    check_route(l, k, scores=scores, groups=groups, top_groups=top, group_best=best, bias=bias)


def test_route_scores_a_few_parts_in_two_to_the_24_apart():
    """Choice values that fp32 cannot tell apart are chosen as in double precision."""
    need_gpu()
    r = np.random.default_rng(1)
    T, E = 200, 64
    l = torch.from_numpy(r.standard_normal((T, E))).float().cuda()
    s = 1 / (1 + np.exp(-as64(l)))
    # one token's scores are all brought to 1 by the bias, up to fp32's rounding of it
    bias = torch.from_numpy(1 - s[0]).float().cuda()
    check_route(l, 8, scores="sigmoid", bias=bias)
    check_route(l, 8, scores="sigmoid", bias=bias, groups=8, top_groups=3, group_best=2)
    assert len(set(np.float32(as64(bias) + s[0]).tolist())) < 8


def test_route_infinite_and_extreme_logits():
    need_gpu()
    inf = float("inf")
    l = torch.randn(12, 16, device="cuda")
    l[0, 3] = inf
    l[1, 3] = l[1, 9] = inf
    l[2] = inf
    l[3] = -1000.0      # sigmoid and exp vanish
    l[4] = 1000.0
    l[5] = torch.tensor([-1000.0] * 8 + [1000.0] * 8)
    l[6] = -inf
    l[7] = float("nan")
    l[8, ::2] = -3e38
    bias = torch.randn(16, device="cuda")
    bias[2], bias[5] = -inf, float("nan")
    for how in (dict(), dict(groups=4, top_groups=2, group_best=2)):
        for scores in ("softmax", "sigmoid"):
            for renormalize in (True, False):
                check_route(l, 4, scores=scores, renormalize=renormalize, **how)
                check_route(l, 4, scores=scores, renormalize=renormalize, bias=bias, **how)


def test_route_empty_strided_and_unsorted():
    need_gpu()
    l = logits_of(0, 8, "f32", 1, False)
    w, e, rows, pos, off = w4.w4a4_route_experts_scored(l, 2, scores="sigmoid", groups=4, top_groups=2)
    assert w.shape == (0, 2) and rows.shape == (0,) and bool((off == 0).all())
    wide = logits_of(50, 100, "bf16", 2)
    check_route(wide[:, 3:35], 4, scores="sigmoid", groups=4, top_groups=2)


def test_route_equals_plain_routing():
    """Softmax without a bias or groups is w4a4_route_experts' choice."""
    need_gpu()
    l = logits_of(500, 64, "f32", 4)
    for renormalize in (True, False):
        a = w4.w4a4_route_experts(l, 6, renormalize=renormalize)
        b = w4.w4a4_route_experts_scored(l, 6, renormalize=renormalize)
        assert all(torch.equal(x, y) for x, y in zip(a[1:], b[1:]))
        assert bool(((a[0] - b[0]).abs() <= 2.0 ** -20 * b[0]).all())   # fp32 exp and sums of 64


# ---- the layer ------------------------------------------------------------------

def layer(E, K, F, h, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    w13 = w4.w8a8_quantize_weights_fp8(torch.randn(E, 2 * F, K, device="cuda", generator=g) * K ** -0.5, h)
    w2 = w4.w8a8_quantize_weights_fp8(torch.randn(E, K, F, device="cuda", generator=g) * F ** -0.5)
    return (*w13, *w2)


HOW = dict(scores="sigmoid", groups=4, top_groups=2, group_best=2, renormalize=True, scale=2.5)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("T,g", [(1, 0), (16, 64), (150, 32), (900, 0)])
def test_experts_are_their_parts(T, g, dtype):
    need_gpu()
    E, K, F, k = 8, 384, 256, 3
    h = w4.Hadamard(g, *signs(g, 2)) if g else None
    w = layer(E, K, F, h)
    x, l = draw_x(T, K, dtype, T), logits_of(T, E, "f32", T, T > 20)
    bias = 0.1 * torch.randn(E, device="cuda")
    weights, experts, rows, pos, off = w4.w4a4_route_experts_scored(l, k, bias=bias, **HOW)
    codes, scales = w4.w8a8_quantize_fp8(x, h)
    hc, hs = w4.w8a8_grouped_gated_fp8(codes, scales, w[0], w[1], off, rows=rows)
    for rd in {DT[dtype], torch.float32}:
        y = w4.w8a8_grouped_gemm_fp8(hc, hs, w[2], w[3], off, out_dtype=rd)
        want = w4.w4a4_combine_experts(y, pos, weights, out_dtype=DT[dtype])
        got = w4.w8a8_experts_fp8(x, l, k, *w, h=h, bias=bias, rows_dtype=rd, **HOW)
        if rd == DT[dtype]:
            assert torch.equal(got, want)
            continue
        # The layer takes the fp8 matrix core for a 16-bit x whatever its rows' type, the
        # part with fp32 outputs the fp16 one: they differ by the former's bound, weighted,
        # and each side rounds to the output's type (and sums in fp32).
        act, at = fp8.values(raw(hc), as64(hs).T), off.cpu().numpy()
        w2 = fp8.values(raw(w[2]), as64(w[3]), 128)
        room = np.zeros((T, K))
        for e in range(E):
            rows_e = np.arange(at[e], at[e + 1])
            b = fp8.product_bound(act[rows_e], w2[e]) + 2.0 ** -22 * np.abs(act[rows_e]) @ np.abs(w2[e]).T
            token, choice = np.nonzero(np.isin(pos.cpu().numpy(), rows_e))
            order = pos.cpu().numpy()[token, choice] - at[e]
            np.add.at(room, token, np.abs(as64(weights))[token, choice][:, None] * b[order])
        rel, step = mx4.HALF_ULP[dtype]
        assert (np.abs(as64(got) - as64(want)) <= room + 2 * rel * (np.abs(as64(want)) + room) + 2 * step).all()


def test_experts_against_64_bits():
    """The layer on fp32 data against its definition: the activations' codes are the
    quantiser's, the experts' inner codes may move by one where fp32 sums put a value
    on the other side of a border (1 in 16 of the value, of a block's 448 steps)."""
    need_gpu()
    T, E, K, F, k = 40, 4, 256, 128, 2
    w = layer(E, K, F, None)
    x, l = draw_x(T, K, "f32", 1), logits_of(T, E, "f32", 1, False)
    got = as64(w4.w8a8_experts_fp8(x, l, k, *w, scores="sigmoid"))
    weights, experts, *_ = fp8.route(as64(l), k, scores="sigmoid")
    codes, scales = w4.w8a8_quantize_fp8(x)
    av = fp8.values(raw(codes), as64(scales).T)
    w13, w2 = fp8.values(raw(w[0]), as64(w[1]), 128), fp8.values(raw(w[2]), as64(w[3]), 128)
    ref, room = np.zeros((T, K)), np.zeros((T, K))
    for t in range(T):
        for j in range(k):
            e = experts[t, j]
            y, err = w13[e] @ av[t], fp8.product_bound(av[t:t + 1], w13[e], "f32")[0]
            g, u = y[:F], y[F:]
            v = fp8.silu(g) * u
            eps = 1.1 * np.abs(u) * err[:F] + np.abs(fp8.silu(g)) * err[F:] + (np.abs(g) + 5) * 2.0 ** -23 * np.abs(v)
            c, s = fp8.quantize(v[None])
            act = fp8.values(c, s)
            lo, hi = (fp8.GRID[fp8.nearest_code(np.maximum(np.abs(v) + d * (eps + 2.0 ** -21 * np.abs(v)), 0) / s[0, 0])] for d in (-1, 1))
            moved = (hi - lo) * s[0, 0] + 2.0 ** -20 * np.abs(act[0])
            ref[t] += weights[t, j] * (w2[e] @ act[0])
            room[t] += weights[t, j] * (np.abs(w2[e]) @ moved + fp8.product_bound(act, w2[e])[0] + 2.0 ** -22 * np.abs(w2[e] @ act[0]))
    assert (np.abs(got - ref) <= room).all()


def test_experts_padding_and_single_expert():
    need_gpu()
    w = layer(1, 128, 128, None)
    x = draw_x(5, 128, "bf16", 1)
    l = torch.zeros(5, 1, device="cuda")
    l[2] = -float("inf")
    got = w4.w8a8_experts_fp8(x, l, 1, *w)
    assert bool((got[2] == 0).all()) and bool((got[0] != 0).any())
    assert w4.w8a8_experts_fp8(x[:0], l[:0], 1, *w).shape == (0, 128)
    assert w4.w8a8_experts_fp8(x.view(1, 5, 128), l, 1, *w).shape == (1, 5, 128)


def test_experts_captured():
    """Two graphs with workspaces of their own, replayed in turn with new inputs."""
    need_gpu()
    E, K, F, k = 8, 256, 128, 2
    w = layer(E, K, F, None)
    bias = 0.1 * torch.randn(E, device="cuda")
    held = []
    for T in (3, 200):
        x, l = draw_x(T, K, "bf16", T), logits_of(T, E, "f32", T, False)
        ws = torch.empty(w4.w8a8_experts_fp8_workspace_size(T, K, F, E, k, torch.float32), dtype=torch.uint8, device="cuda")
        w4.w8a8_experts_fp8(x, l, k, *w, bias=bias, workspace=ws, **HOW)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = w4.w8a8_experts_fp8(x, l, k, *w, bias=bias, workspace=ws, **HOW)
        held.append((graph, x, l, out))
    for i in range(4):
        for graph, x, l, out in held:
            x.mul_(-1.5)
            l.copy_(l.roll(1, 1))
            graph.replay()
            want = w4.w8a8_experts_fp8(x, l, k, *w, bias=bias, **HOW)
            torch.cuda.synchronize()
            assert torch.equal(out, want)

"""GPU tests of the MX4 operators where the other files do not go: the skinny kernels
that split a long K over eight waves, calls under graph capture, strided activations
through the layers, row numbers outside the codes through the gated product, gates far
below zero."""
import numpy as np
import pytest
import torch

from tests import mx4
from tests.gpu_util import need_gpu
from tests.test_gpu_mx4 import DT, as64, draw_x, operand, signs
from tests.test_gpu_mx4_experts import check_gated, logits_of, offsets_of

pytestmark = pytest.mark.gpu

import bit_quantized_linear_rotate_amd as w4  # noqa: E402

# K above 1792: eight waves share the steps of one column group (a ragged last step; many steps)
DEEP_K = (1824, 3840)
GROUPS = {
    "one row": ([1], 0),
    "one expert": ([9], 0),
    "up to 16 rows": ([0, 3, 1, 0, 16, 17, 2, 0], 5),
    "up to 32 rows": ([33, 0, 20, 64, 5, 31], 0),
    "up to 64 rows": ([64, 40, 0, 65], 2),
    "nothing routed": ([0, 0, 0], 7),
}


def test_deep_cases_take_the_skinny_kernel():
    for K in DEEP_K:
        for counts, extra in GROUPS.values():
            R, E = sum(counts) + extra, len(counts)
            assert K > 1792 and w4.w4a4_gemm_mx4_plan(R, K, 96, E) == w4.w4a4_gemm_mx4_plan(R, K, 192, E, True) == "skinny"
    # rows a pass, by the mean group: all three
    assert {min(64, 16 << max(0, (-(-(sum(c) + x) // len(c)) - 1) // 16)) for c, x in GROUPS.values()} >= {16, 32, 64}


@pytest.mark.parametrize("name", GROUPS)
@pytest.mark.parametrize("K", DEEP_K)
def test_deep_grouped_gemm(name, K):
    need_gpu()
    counts, extra = GROUPS[name]
    E, R, N = len(counts), sum(counts) + extra, 96
    T = max(1, R // 2)
    a, sa, av = operand(T, K, 1)
    w, sw, wv = operand(N, K, 2, (E,))
    rows = np.random.default_rng(R).integers(0, T, R).astype(np.int32)
    off = offsets_of(counts)
    o = off.cpu().numpy()
    b = torch.randn(E, N, device="cuda").to(torch.bfloat16)
    ref, bound = np.zeros((R, N)), np.zeros((R, N))
    for e in range(E):
        at = slice(o[e], o[e + 1])
        x = av[rows[at]]
        ref[at] = x @ wv[e].T + as64(b[e])
        bound[at] = mx4.product_bound(x, wv[e]) + 2.0 ** -24 * (np.abs(ref[at]) + 2 * np.abs(as64(b[e])))
    for out in DT:
        got = w4.w4a4_grouped_gemm_mx4(a, sa, w, sw, off, rows=torch.from_numpy(rows).cuda(), bias=b, out_dtype=DT[out])
        mx4.close(as64(got), ref, bound, out)
        assert bool((got[o[E]:] == 0).all())


@pytest.mark.parametrize("name", GROUPS)
@pytest.mark.parametrize("K", DEEP_K)
def test_deep_grouped_gated(name, K):
    need_gpu()
    counts, extra = GROUPS[name]
    E, R, F = len(counts), sum(counts) + extra, 96
    T = max(1, R // 2)
    a, sa, av = operand(T, K, 1)
    w, sw, wv = operand(2 * F, K, 2, (E,))
    sa = (sa.int() - 6).clamp(min=0).to(torch.uint8)
    av = av * 2.0 ** -6
    rows = np.random.default_rng(R).integers(0, T, R).astype(np.int32)
    rows[R // 2:R // 2 + 1] = -1                           # rows that are not there: silu(0) * 0
    rows[R // 3:R // 3 + 1] = T
    off = offsets_of(counts)
    o = off.cpu().numpy()
    codes, scales = w4.w4a4_grouped_gated_mx4(a, sa, w, sw, off, rows=torch.from_numpy(rows).cuda())
    codes, full = codes.cpu().numpy(), scales.cpu().numpy()
    srows = mx4.unslab(full, F)
    assert np.array_equal(full, mx4.slabs(srows)) and not codes[o[E]:].any() and not srows[o[E]:].any()
    for e in range(E):
        at = slice(o[e], o[e + 1])
        if o[e] == o[e + 1]:
            continue
        x = np.where(((rows[at] >= 0) & (rows[at] < T))[:, None], av[np.clip(rows[at], 0, T - 1)], 0)
        y, bound = x @ wv[e].T, mx4.product_bound(x, wv[e])
        check_gated(codes[at], srows[at], y[:, :F], y[:, F:], bound[:, :F], bound[:, F:])


@pytest.mark.parametrize("M,K,N", [(20, 1824, 96), (32, 3840, 4000), (33, 3840, 96), (64, 2080, 513)])
def test_deep_dense(M, K, N):
    need_gpu()
    a, sa, av = operand(M, K, 1)
    w, sw, wv = operand(N, K, 2)
    assert w4.w4a4_gemm_mx4_plan(M, K, N) == "skinny"
    for out in DT:
        got = w4.w4a4_gemm_mx4(a, sa, w, sw, out_dtype=DT[out])
        mx4.close(as64(got), av @ wv.T, mx4.product_bound(av, wv), out)


@pytest.mark.parametrize("counts", [[9, 4], [200, 150], [700, 400]])
def test_gated_rows_outside_the_codes(counts):
    need_gpu()
    R, T, K, F = sum(counts), 50, 256, 96
    a, sa, _ = operand(T, K, 1)
    w, sw, _ = operand(2 * F, K, 2, (2,))
    sa = (sa.int() - 5).clamp(min=0).to(torch.uint8)
    rows = np.random.default_rng(1).integers(0, T, R).astype(np.int32)
    gone = [3, 5, R - 1]
    inside = torch.from_numpy(rows).cuda()
    ref = w4.w4a4_grouped_gated_mx4(a, sa, w, sw, offsets_of(counts), rows=inside)
    rows[gone] = -1, 2 ** 31 - 1, T
    got = w4.w4a4_grouped_gated_mx4(a, sa, w, sw, offsets_of(counts), rows=torch.from_numpy(rows).cuda())
    keep = np.setdiff1d(np.arange(R), gone)
    assert torch.equal(got[0][keep], ref[0][keep]) and torch.equal(got[1][:, keep], ref[1][:, keep])
    assert not bool((got[0][gone] & 0x77).any()) and not bool(got[1][:, gone].any())   # zeros of either sign


def exact_sums(target):
    """Codes of 32 values that add up to each integer of target (at most 384 in
    magnitude), as multiples of 1 under the scale 2: every partial sum is exact."""
    flat = target.reshape(-1)
    mag = (mx4.GRID * 2).astype(np.int64)
    n = np.zeros((flat.size, 32), np.uint8)
    left = np.abs(flat).astype(np.int64)
    for i in range(32):
        c = np.searchsorted(mag, left, side="right") - 1
        left = left - mag[c]
        n[:, i] = c | np.where((flat < 0) & (c > 0), 8, 0)
    assert not left.any()
    return (n[:, 0::2] | (n[:, 1::2] << 4)).reshape(*target.shape, 16)


@pytest.mark.parametrize("R", [5, 300, 2000])
def test_gates_far_below_zero(R):
    """Gates from -96 to 96, each block's alike, with sums that are exact, so all the error
    is the activation's.  exp is 2^(g log2(e)), whose argument is rounded twice (2 |g| 2^-24
    of the result) and whose power is good to one unit, like the reciprocal (2^-23 each);
    three roundings (2^-24 each): (|g| + 4) 2^-23 of the value.  The reciprocal is zero
    below 2^-126: |g u| 2^-126; the products' smallest steps."""
    need_gpu()
    F = 32 * 49
    r = np.random.default_rng(R)
    g = np.repeat(np.arange(-96, 97, 4), 32) + r.integers(-1, 2, F)
    u = r.integers(1, 300, F) * r.choice([-1, 1], F)
    w = exact_sums(np.concatenate([g, u])[None])
    sw = mx4.slabs(np.full((1, 2 * F, 1), 128, np.uint8))
    a = np.full((R, 16), 0x22, np.uint8)                   # ones
    half = r.integers(0, 2, R)                             # under scales 1 and 1/2
    sa = mx4.slabs((127 - half)[:, None].astype(np.uint8))
    cuda = lambda t: torch.from_numpy(t).cuda()  # noqa: E731
    codes, scales = w4.w4a4_grouped_gated_mx4(cuda(a), cuda(sa), cuda(w), cuda(sw), offsets_of([R]))
    gr, ur = g * 0.5 ** half[:, None], u * 0.5 ** half[:, None]
    v = mx4.silu(gr) * ur
    err = (np.abs(gr) + 4) * 2.0 ** -23 * np.abs(v) + np.abs(gr * ur) * 2.0 ** -126 + 2.0 ** -147
    srows = mx4.unslab(scales.cpu().numpy(), F)
    got = mx4.values(codes.cpu().numpy(), srows).reshape(R, -1, 32)
    blocks = lambda t: t.reshape(R, -1, 32)  # noqa: E731
    lo, hi = blocks(np.maximum(np.abs(v) - err, 0)), blocks(np.abs(v) + err)
    X = srows.astype(np.int64) - 127
    assert (X >= mx4.scale_exponent(lo.max(-1))).all() and (X <= mx4.scale_exponent(hi.max(-1))).all()
    s = np.exp2(X.astype(np.float64))[..., None]
    m = np.abs(got) / s
    assert (m >= mx4.GRID[mx4.nearest_code(lo / s)]).all() and (m <= mx4.GRID[mx4.nearest_code(hi / s)]).all()
    assert (np.signbit(got) == np.signbit(blocks(v)))[got != 0].all()


def test_strided_activations_through_the_layers():
    need_gpu()
    M, K, N, F, E, g = 70, 512, 96, 64, 4, 64
    _, sid = signs(g, 1)
    h = w4.Hadamard(g, sid)
    x = draw_x(M, K, "bf16", 1)
    w, sw, _ = operand(N, K, 2)
    w13, s13, _ = operand(2 * F, K, 3, (E,))
    w2, s2, _ = operand(K, F, 4, (E,))
    l = logits_of(M, E, "bf16", 5)
    wide = torch.zeros((M, K + 11), dtype=x.dtype, device="cuda")
    wide[:, 5:K + 5] = x
    many = torch.zeros((M, 2 * E), dtype=l.dtype, device="cuda")
    many[:, 1:E + 1] = l
    ref = w4.w4a4_linear_mx4(x, w, sw, h=h), w4.w4a4_experts_mx4(x, l, 2, w13, s13, w2, s2, h=h)
    for v in (x.t().contiguous().t(), wide[:, 5:K + 5], torch.stack([x, x], 1)[:, 1]):
        assert torch.equal(w4.w4a4_linear_mx4(v, w, sw, h=h), ref[0])
        assert torch.equal(w4.w4a4_experts_mx4(v, many[:, 1:E + 1], 2, w13, s13, w2, s2, h=h), ref[1])


@pytest.mark.parametrize("E,k", [(8, 2), (300, 20)])
def test_route_infinite_logits(E, k):
    """An infinite logit is taken first, and leaves no weights; the lowest finite value is a
    logit like others, and a row of them an even one."""
    need_gpu()
    l = logits_of(40, E, "f32", 1)
    l[7, 3] = l[9, 2] = l[9, 5] = float("inf")
    l[11], l[12] = torch.finfo(torch.float32).min, float("-inf")
    l[12, 4] = torch.finfo(torch.float32).min
    for renorm in (True, False):
        w, e, rows, pos, off = (t.cpu() for t in w4.w4a4_route_experts(l, k, renormalize=renorm))
        assert e[7, 0] == 3 and e[9, :2].tolist() == [2, 5] and w[7].isnan().all() and w[9].isnan().all()
        assert e[11].tolist() == list(range(k)) and torch.equal(w[11], torch.full((k,), 1 / (k if renorm else E)))
        assert e[12].tolist() == [4] + [-1] * (k - 1) and w[12].tolist() == [1.0] + [0.0] * (k - 1)
        others = [t for t in range(40) if t not in (7, 9)]
        ref = mx4.route(as64(l[others]), k, renorm)
        assert np.array_equal(e[others].numpy(), ref[1])
        assert (np.abs(w[others].double().numpy() - ref[0]) <= (E + 64) * 2.0 ** -24 * ref[0]).all()


@pytest.mark.parametrize("T", [16, 300])
def test_routing_and_layer_replay_in_a_graph(T):
    """T = 300: routing in several chunks, two launches."""
    need_gpu()
    K, F, E, k = 256, 64, 8, 2
    x, l = draw_x(T, K, "bf16", 1), logits_of(T, E, "f32", 2)
    w13, s13, _ = operand(2 * F, K, 3, (E,))
    w2, s2, _ = operand(K, F, 4, (E,))
    s13 = (s13.int() - 6).clamp(min=0).to(torch.uint8)
    ws = torch.empty(w4.w4a4_experts_mx4_workspace_size(T, K, F, E, k, torch.bfloat16), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(x)

    def calls(**into):
        routed = w4.w4a4_route_experts(l, k)
        codes, scales = w4.w4a4_quantize_mx4(x)
        hidden = w4.w4a4_grouped_gated_mx4(codes, scales, w13, s13, routed[4], rows=routed[2])
        y = w4.w4a4_grouped_gemm_mx4(*hidden, w2, s2, routed[4], out_dtype=torch.float32)
        both = w4.w4a4_combine_experts(y, routed[3], routed[0])
        return (*routed, both, w4.w4a4_experts_mx4(x, l, k, w13, s13, w2, s2, **into))

    calls(workspace=ws, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = calls(workspace=ws, out=out)
    for seed in range(4):
        x.copy_(draw_x(T, K, "bf16", 20 + seed))
        l.copy_(logits_of(T, E, "f32", 30 + seed))
        ref = calls()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        # (rows past the last routed one are -1 in both, positions that are none -1)
        for i, (a, b) in enumerate(zip(held, ref)):
            assert torch.equal(a, b), (seed, i)

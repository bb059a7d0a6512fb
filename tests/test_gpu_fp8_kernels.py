"""GPU tests of the fp8 products' and of scored routing's kernels that sizes alone select:
every variant by name, outputs that are exact, many tiles a workgroup, wide rows, many
tokens."""
import numpy as np
import pytest
import torch

from tests import fp8
from tests.gpu_util import need_gpu
from tests.test_gpu_fp8 import DT, F8, as64, raw, rows_operand, weights_operand

pytestmark = pytest.mark.gpu

import bit_quantized_linear_rotate_amd as w4  # noqa: E402


@pytest.fixture(autouse=True)
def seeded():
    torch.manual_seed(7)


# Codes of integers up to 4 under powers of two from 2^-1 to 2: products up to 16, sums
# of eight 128 (any fixed point of 13 bits below the largest holds them), blocks up to
# 2^11, scales' products quarters to 4; sums of up to 2^22 quarters, so every order of
# fp32 sums is exact and the outputs are the exact ones rounded once.
def ints(*shape):
    return torch.randint(-4, 5, shape, device="cuda").float()


def powers(*shape):
    return 2.0 ** torch.randint(-1, 2, shape, device="cuda").float()


def rows_of_ints(M, K):
    """(codes, scales, values) of rows, values float64."""
    v, s = ints(M, K), powers(fp8.blocks(K), M)
    return v.to(F8), s, (v * s.t().repeat_interleave(128, 1)[:, :K]).double()


def weights_of_ints(N, K, E=1):
    v, s = ints(E, N, K), powers(E, fp8.blocks(N), fp8.blocks(K))
    full = s.repeat_interleave(128, 1)[:, :N].repeat_interleave(128, 2)[..., :K]
    return v.to(F8), s, (v * full).double()


# what a call's sizes select: rows, K, N -> kernel of 16-bit outputs; the skinny ones by
# row tiles, column tiles (2: more than 512 groups of 16 columns) and waves a column group
SKINNY = [(1, 16, 48, "1 1 4"), (9, 1040, 300, "1 1 8"), (20, 400, 130, "2 1 4"), (20, 1040, 2001, "2 1 8"),
          (64, 272, 1000, "4 1 4"), (50, 1040, 513, "4 1 8"), (1, 16, 8209, "1 2 4"), (3, 1040, 10257, "1 2 8"),
          (17, 400, 8209, "2 2 4"), (32, 1040, 8300, "2 2 8"), (33, 144, 8209, "4 2 4"), (64, 1040, 8335, "4 2 8"),
          (100, 528, 8209, "4 2 4")]


def skinny_variant(M, K, N):
    """The skinny kernel's row tiles, column tiles and waves a column group."""
    rows = 16 if M <= 16 else 32 if M <= 32 else 64
    groups = -(-N // 16) * -(-M // rows)
    return f"{rows // 16} {1 if groups <= 512 else 2} {8 if K > 1024 else 4}"


def test_skinny_sizes_reach_every_variant():
    assert {v for *_, v in SKINNY} == {f"{m} {n} {k}" for m in (1, 2, 4) for n in (1, 2) for k in (4, 8)}
    for M, K, N, variant in SKINNY:
        assert w4.w8a8_gemm_fp8_plan(M, K, N) == "skinny" and skinny_variant(M, K, N) == variant, (M, K, N)


@pytest.mark.parametrize("M,K,N", [s[:3] for s in SKINNY])
def test_skinny_variants(M, K, N):
    need_gpu()
    a, sa, av = rows_of_ints(M, K)
    w, sw, wv = weights_of_ints(N, K)
    ref = av @ wv[0].t()
    b = ints(N)
    for out in DT:
        assert torch.equal(w4.w8a8_gemm_fp8(a, sa, w[0], sw[0], out_dtype=DT[out]), ref.to(DT[out]))
        got = w4.w8a8_gemm_fp8(a, sa, w[0], sw[0], bias=b.to(DT[out]), out_dtype=DT[out])
        assert torch.equal(got, (ref + b.double()).to(DT[out]))
    a, sa, av = rows_operand(M, K, M)
    w, sw, wv = weights_operand(N, K, N)
    got = as64(w4.w8a8_gemm_fp8(a, sa, w, sw, out_dtype=torch.float32))
    ref = av @ wv.T
    assert (np.abs(got - ref) <= fp8.product_bound(av, wv, "f32") + 2.0 ** -24 * np.abs(ref)).all()


# Outputs of 8 MB a row and more, which tiles cannot address: the skinny kernel, whatever
# the rows.
@pytest.mark.parametrize("M,N,out", [(1, 2 ** 21 + 1, "f32"), (150, 2 ** 21 + 1, "f32"), (150, 2 ** 22, "bf16")])
def test_outputs_of_8_mb_a_row(M, N, out):
    need_gpu()
    K = 16
    if out == "bf16":
        assert w4.w8a8_gemm_fp8_plan(M, K, N) == "skinny"
    a, sa, av = rows_of_ints(M, K)
    w, sw, wv = weights_of_ints(N, K)
    got = w4.w8a8_gemm_fp8(a, sa, w[0], sw[0], out_dtype=DT[out])
    for m in range(0, M, 50):   # (sums of 16 exact terms: fp32 holds them)
        assert torch.equal(got[m:m + 50], (av[m:m + 50].float() @ wv[0].float().t()).to(DT[out]))


# More than 128 tiles for each of 256 workgroups: the list of a workgroup's tiles is
# filled three times, the third over the first.
@pytest.mark.parametrize("out,M,N", [("bf16", 999983, 2304), ("f16", 980001, 2311), ("f32", 700001, 1793)])
def test_many_dense_tiles_a_workgroup(out, M, N):
    need_gpu()
    K = 16
    rows = 128 if out == "f32" else 256
    assert -(-M // rows) * -(-N // 256) > 128 * 256
    if out != "f32":
        assert w4.w8a8_gemm_fp8_plan(M, K, N) == "tile256"
    a, sa, av = rows_of_ints(M, K)
    w, sw, wv = weights_of_ints(N, K)
    got = w4.w8a8_gemm_fp8(a, sa, w[0], sw[0], out_dtype=DT[out])
    wt = wv[0].float().t().contiguous()
    for m in range(0, M, 1 << 16):
        assert torch.equal(got[m:m + (1 << 16)], (av[m:m + (1 << 16)].float() @ wt).to(DT[out])), m


def test_an_output_of_64_gb():
    """2^20 x 32768 bf16: offsets past 2^35, 2048 tiles for each workgroup."""
    need_gpu()
    M, K, N = 1 << 20, 16, 1 << 15
    if torch.cuda.mem_get_info()[0] < 100 << 30:
        pytest.skip("less than 100 GB of free memory")
    a, sa, av = rows_of_ints(M, K)
    w, sw, wv = weights_of_ints(N, K)
    got = w4.w8a8_gemm_fp8(a, sa, w[0], sw[0])
    wt = wv[0].float().t().contiguous()
    for m in range(0, M, 1 << 14):
        assert torch.equal(got[m:m + (1 << 14)], (av[m:m + (1 << 14)].float() @ wt).bfloat16()), m
    del got
    torch.cuda.empty_cache()


def test_many_grouped_tiles_a_workgroup():
    """16384 experts of one or two rows, three column tiles each; the gated product
    against the same experts in eight calls of few tiles."""
    need_gpu()
    E, K, N = 16384, 32, 768
    counts = np.arange(E) % 2 + 1
    R = int(counts.sum())
    assert w4.w8a8_gemm_fp8_plan(R, K, N, E) == w4.w8a8_gemm_fp8_plan(R, K, N, E, True) == "tile64"
    off = np.concatenate([[0], np.cumsum(counts)])
    offsets = torch.from_numpy(off.astype(np.int32)).cuda()
    expert = torch.from_numpy(np.repeat(np.arange(E), counts)).cuda()
    a, sa, av = rows_of_ints(R, K)
    w, sw, wv = weights_of_ints(N, K, E)
    ref = torch.cat([(wv[expert[i:i + 1024]] * av[i:i + 1024, None]).sum(2) for i in range(0, R, 1024)])
    for out in DT:
        assert torch.equal(w4.w8a8_grouped_gemm_fp8(a, sa, w, sw, offsets, out_dtype=DT[out]), ref.to(DT[out]))
    w, sw, _ = weights_operand(N, K, 2, 8)
    w, sw = w.view(torch.uint8).repeat(E // 8, 1, 1).view(F8), sw.repeat(E // 8, 1, 1)
    codes, scales = w4.w8a8_grouped_gated_fp8(a, sa, w, sw, offsets)
    for e in range(0, E, E // 8):
        r = slice(off[e], off[e + E // 8])
        part = offsets[e:e + E // 8 + 1] - offsets[e]
        c, s = w4.w8a8_grouped_gated_fp8(a[r], sa[:, r].contiguous(), w[e:e + E // 8], sw[e:e + E // 8], part)
        assert torch.equal(codes[r].view(torch.uint8), c.view(torch.uint8)) and torch.equal(scales[:, r], s)


# counts per expert, rows that no expert owns before and behind, K, N, kernel
GROUPED = [([33, 0, 20, 64, 5, 31], 0, 3, 1040, 2561, "tile64"), ([3, 64, 40, 0, 33, 1, 64, 17] * 8, 5, 2, 144, 130, "tile64"),
           ([128, 129, 0, 600, 255, 1], 2, 9, 1040, 3330, "tile128"), ([300, 500, 0, 129] * 2, 0, 0, 272, 2051, "tile128"),
           ([256, 2049, 0, 513, 1, 700], 1, 1, 1040, 2561, "tile256"), ([2600, 1, 2049, 513], 7, 2, 144, 2304, "tile256")]


@pytest.mark.parametrize("counts,before,behind,K,N,kernel", GROUPED)
@pytest.mark.parametrize("gather", [False, True])
def test_grouped_outputs_are_exact(counts, before, behind, K, N, kernel, gather):
    need_gpu()
    E, R = len(counts), sum(counts) + before + behind
    assert w4.w8a8_gemm_fp8_plan(R, K, N, E) == kernel
    M = R // 2 + 1 if gather else R
    a, sa, av = rows_of_ints(M, K)
    w, sw, wv = weights_of_ints(N, K, E)
    rows = torch.randint(0, M, (R,), device="cuda", dtype=torch.int32) if gather else None
    if gather:
        rows[before], rows[R - behind - 1] = M, -1   # no such rows: zeros
    off = np.concatenate([[0], np.cumsum(counts)]) + before
    b = ints(E, N)
    ref = torch.zeros(R, N, device="cuda", dtype=torch.float64)
    for e in range(E):
        at = slice(off[e], off[e + 1])
        x = av[at]
        if gather:
            r = rows[at].long()
            x = torch.where(((r >= 0) & (r < M))[:, None], av[r.clamp(0, M - 1)], 0.0)
        ref[at] = x @ wv[e].t() + b[e].double()
    owned = torch.zeros(R, 1, device="cuda", dtype=torch.bool)
    owned[off[0]:off[E]] = True
    bare = torch.where(owned, ref - torch.repeat_interleave(
        torch.cat([torch.zeros(1, N, device="cuda"), b, torch.zeros(1, N, device="cuda")]).double(),
        torch.tensor([before, *counts, behind], device="cuda"), 0), 0.0)
    offsets = torch.from_numpy(off.astype(np.int32)).cuda()
    for out in DT:
        got = w4.w8a8_grouped_gemm_fp8(a, sa, w, sw, offsets, rows=rows, bias=b, out_dtype=DT[out])
        assert torch.equal(got, ref.to(DT[out]))
        assert torch.equal(w4.w8a8_grouped_gemm_fp8(a, sa, w, sw, offsets, rows=rows, out_dtype=DT[out]), bare.to(DT[out]))


# tokens, experts, K, F, kernel of the second product
LAYERS = [(40, 8, 272, 128, "tile64"), (600, 4, 3600, 384, "tile128"), (900, 4, 2320, 128, "tile128"),
          (1500, 4, 3600, 384, "tile256"), (6000, 3, 2320, 128, "tile256")]


@pytest.mark.parametrize("T,E,K,F,kernel", LAYERS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_layer_with_fp32_rows_of_every_tile(T, E, K, F, kernel, dtype):
    """16-bit activations, rows kept in fp32: the layer's second product comes from the
    fp8 matrix core, its parts' from the fp16 one.  Where every product and sum is exact
    both are the same to the bit: gates of 64 (silu(64) is 64 in fp32) and ups of 0, +-1,
    +-2 and +-4 have the codes 112 |up| under their block's largest or its half, a quarter,
    whatever the roundings of their sums, and the second weights' codes are integers."""
    need_gpu()
    k = 2
    assert w4.w8a8_gemm_fp8_plan(T * k, F, K, E) == kernel
    pick = torch.tensor([0.0, 1.0, 2.0, 4.0], device="cuda")
    x = pick[torch.randint(0, 4, (T, K), device="cuda")] * (torch.randint(0, 2, (T, K), device="cuda") * 2 - 1).float()
    x[:, ::128] = 4.0                                    # every block's scale is 4 / 448
    w13 = torch.zeros(E, 2 * F, K, device="cuda")
    w13[:, :F, 0] = 16.0                                 # gates 64
    for e in range(E):                                   # ups: a value of the token each
        w13[e, F + torch.arange(F, device="cuda"), torch.randint(1, K, (F,), device="cuda")] = 1.0
    w13c, w13s = w4.w8a8_quantize_weights_fp8(w13)
    w2c, w2s, _ = weights_of_ints(K, F, E)
    l = torch.randn(T, E, device="cuda")
    weights, experts, rows, pos, off = w4.w4a4_route_experts_scored(l, k)
    codes, scales = w4.w8a8_quantize_fp8(x.to(DT[dtype]))
    hc, hs = w4.w8a8_grouped_gated_fp8(codes, scales, w13c, w13s, off, rows=rows)
    mags = raw(hc) & 127
    assert set(np.unique(fp8.GRID[mags])) <= {0.0, 112.0, 224.0, 448.0}
    y = w4.w8a8_grouped_gemm_fp8(hc, hs, w2c, w2s, off, out_dtype=torch.float32)
    want = w4.w4a4_combine_experts(y, pos, weights, out_dtype=DT[dtype])
    got = w4.w8a8_experts_fp8(x.to(DT[dtype]), l, k, w13c, w13s, w2c, w2s)
    assert torch.equal(got, want) and bool((got != 0).any())


# ---- routing by scores -----------------------------------------------------------

@pytest.mark.parametrize("T,E,k,groups,top_groups", [(70, 128, 8, 8, 3), (20, 96, 6, 4, 2), (33, 66, 14, 11, 4), (5, 128, 14, 64, 20)])
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_route_groups_of_65_to_128_experts(T, E, k, groups, top_groups, scores):
    from tests.test_gpu_fp8_experts import check_route, logits_of
    need_gpu()
    bias = torch.from_numpy(0.2 * np.random.default_rng(E).standard_normal(E)).float().cuda()
    how = dict(scores=scores, groups=groups, top_groups=top_groups)
    for dtype in DT:
        l = logits_of(T, E, dtype, T + E)
        check_route(l, k, group_best=1, renormalize=True, **how)
        check_route(l, k, group_best=2, renormalize=False, scale=2.5, **how)
        check_route(l, k, group_best=2, renormalize=True, scale=2.5, bias=bias, **how)
        check_route(l, k, group_best=1, renormalize=False, bias=bias, **how)


def route_finite(l, k, scores, bias, groups, top_groups, group_best):
    """(weights renormalised, experts) of finite logits, 64 bits, all tokens at once."""
    T, E = l.shape
    l = l.double()
    s = torch.sigmoid(l) if scores == "sigmoid" else torch.softmax(l, 1)
    v = s if bias is None else s + bias.double()
    order = l if bias is None else v
    if top_groups < groups:
        of = (l if bias is None and group_best == 1 else v).view(T, groups, E // groups)
        worth = of.topk(min(group_best, E // groups), 2).values.sum(2)
        kept = worth.argsort(dim=1, descending=True, stable=True)[:, :top_groups]
        live = torch.zeros(T, groups, dtype=torch.bool, device=l.device).scatter_(1, kept, True)
        order = order.masked_fill(~live.repeat_interleave(E // groups, 1), -float("inf"))
    experts = order.argsort(dim=1, descending=True, stable=True)[:, :k]
    w = s.gather(1, experts)
    return w / w.sum(1, keepdim=True), experts


# more than 64 tokens a workgroup: its waves take several each, in the variants of few
# experts too
@pytest.mark.parametrize("E,k,groups,top_groups", [(32, 4, 4, 2), (64, 6, 8, 3), (128, 8, 8, 4), (128, 8, 1, 1), (256, 8, 8, 4),
                                                   (256, 20, 4, 2), (512, 10, 16, 5)])
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_route_many_tokens(E, k, groups, top_groups, scores):
    need_gpu()
    T = 20011
    l = torch.randn(T, E, device="cuda")
    bias = 0.2 * torch.randn(E, device="cuda")
    for b, best in ((None, 1), (None, 2), (bias, 2), (bias, 1)):
        want_w, want = route_finite(l, k, scores, b, groups, top_groups, best)
        w, experts, rows, pos, off = w4.w4a4_route_experts_scored(l, k, scores=scores, bias=b, groups=groups,
                                                                  top_groups=top_groups, group_best=best)
        assert torch.equal(experts.long(), want)
        assert bool(((w.double() - want_w).abs() <= (2.0 ** -24 + 2.0 ** -46) * want_w).all())
        flat = want.flatten()
        slots = flat.argsort(dim=0, stable=True)
        assert torch.equal(rows.long(), slots // k)
        assert torch.equal(pos.flatten().long()[slots], torch.arange(T * k, device="cuda"))
        assert torch.equal(off.long()[1:], torch.bincount(flat, minlength=E).cumsum(0)) and int(off[0]) == 0


@pytest.mark.parametrize("E,groups,top_groups,k", [(32, 8, 6, 8), (64, 8, 5, 14), (128, 16, 9, 14), (256, 8, 4, 20)])
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
def test_route_biases_of_the_lowest_value(E, groups, top_groups, k, scores):
    """Experts put last by a bias of the type's lowest value, whole groups of them: the sum
    of a group's two largest is below what fp32 holds, yet a group with such a worth comes
    before one in which nothing can be taken."""
    from tests.test_gpu_fp8_experts import check_route
    need_gpu()
    size, low = E // groups, torch.finfo(torch.float32).min
    l = torch.randn(40, E, device="cuda")
    l[::3, 3 * size:4 * size] = -float("inf")            # a group with nothing to take
    bias = torch.full((E,), low, device="cuda")
    bias[size], bias[2 * size + 1], bias[-1] = 0.25, 0.5, -0.25
    for b in (bias, bias / 2, torch.full_like(bias, low), -bias):
        for best in (1, 2):
            for renormalize in (True, False):
                check_route(l, k, scores=scores, bias=b, groups=groups, top_groups=top_groups, group_best=best,
                            renormalize=renormalize)

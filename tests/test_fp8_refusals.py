"""CPU tests of the fp8 entry points and of routing by scores: every wrong argument is
refused before any device access, by the binding (ValueError) and by the C ABI (status
codes); host-only queries; the plain forms against torch."""
import ctypes
import os
import re

import numpy as np
import pytest
import torch

from bit_quantized_linear_rotate_amd import _binding as b
from tests import fp8

pytestmark = pytest.mark.skipif(not os.path.exists(b.LIB_PATH), reason="libw4a4.so not built")

F8, F32, BF, I32 = torch.float8_e4m3fn, torch.float32, torch.bfloat16, torch.int32
M, K, N, E, F = 6, 304, 48, 4, 128


def z(*shape, dtype=F8):
    return torch.zeros(*shape).to(dtype)


def args(name, **over):
    """Well-formed CPU arguments: refused only for not being on a HIP device."""
    op = dict(codes=z(M, K), scales=z(3, M, dtype=F32))
    w = dict(w_codes=z(N, K), w_scales=z(1, 3, dtype=F32))
    we = dict(w_codes=z(E, 256, K), w_scales=z(E, 2, 3, dtype=F32))
    a = {
        "w8a8_quantize_fp8": dict(x=z(M, K, dtype=BF)),
        "w8a8_quantize_weights_fp8": dict(w=z(E, N, K, dtype=BF)),
        "w8a8_dequantize_fp8": dict(op),
        "w8a8_dequantize_weights_fp8": dict(codes=z(N, K), scales=z(1, 3, dtype=F32)),
        "w8a8_gemm_fp8": dict(op, **w),
        "w8a8_linear_fp8": dict(x=z(M, K, dtype=BF), **w),
        "w8a8_grouped_gemm_fp8": dict(op, **we, offsets=z(E + 1, dtype=I32)),
        "w8a8_grouped_gated_fp8": dict(op, **we, offsets=z(E + 1, dtype=I32)),
        "w4a4_route_experts_scored": dict(logits=z(M, E, dtype=BF), top_k=2),
        "w8a8_experts_fp8": dict(x=z(M, K, dtype=BF), logits=z(M, E, dtype=BF), top_k=2, w13_codes=z(E, 2 * F, K),
                                 w13_scales=z(E, 2, 3, dtype=F32), w2_codes=z(E, K, F), w2_scales=z(E, 3, 1, dtype=F32)),
    }[name]
    a.update(over)
    return a


BAD = [
    ("w8a8_quantize_fp8", dict(x=z(M, 40, dtype=BF)), "multiple of 16"),
    ("w8a8_quantize_fp8", dict(h=b.Hadamard(256)), "multiple of g"),
    ("w8a8_quantize_fp8", dict(h=torch.eye(64)), "Hadamard"),
    ("w8a8_quantize_weights_fp8", dict(w=z(K, dtype=BF)), "expected"),
    ("w8a8_quantize_weights_fp8", dict(w=z(N, 24, dtype=BF)), "multiple of 16"),
    ("w8a8_dequantize_fp8", dict(scales=z(M, 3, dtype=F32)), "scales"),
    ("w8a8_dequantize_fp8", dict(codes=z(M, K).view(torch.uint8)), "dtype"),
    ("w8a8_dequantize_fp8", dict(dtype=torch.float64), "dtype"),
    ("w8a8_dequantize_weights_fp8", dict(scales=z(3, 1, dtype=F32)), "scales"),
    ("w8a8_gemm_fp8", dict(w_codes=z(N, 320)), "w_"),
    ("w8a8_gemm_fp8", dict(w_scales=z(1, 3, dtype=BF)), "dtype"),
    ("w8a8_gemm_fp8", dict(bias=z(N + 1, dtype=BF)), "bias"),
    ("w8a8_gemm_fp8", dict(out_dtype=torch.int8), "out_dtype"),
    ("w8a8_gemm_fp8", dict(codes=z(K, M).t()), "contiguous"),
    ("w8a8_linear_fp8", dict(bias=z(N, dtype=F32)), "bias"),
    ("w8a8_linear_fp8", dict(out=z(M, N + 1, dtype=BF)), "out"),
    ("w8a8_linear_fp8", dict(workspace=z(8).view(torch.uint8)), "workspace|device"),
    ("w8a8_grouped_gemm_fp8", dict(offsets=z(E, dtype=I32)), "offsets"),
    ("w8a8_grouped_gemm_fp8", dict(rows=z(4, dtype=torch.int64)), "rows"),
    ("w8a8_grouped_gemm_fp8", dict(w_codes=z(256, K), w_scales=z(2, 3, dtype=F32)), "dimensions"),
    ("w8a8_grouped_gemm_fp8", dict(bias=z(256, dtype=BF)), "bias"),
    ("w8a8_grouped_gated_fp8", dict(w_codes=z(E, 128, K), w_scales=z(E, 1, 3, dtype=F32)), "blocks of 128"),
    ("w4a4_route_experts_scored", dict(scores="tanh"), "softmax or sigmoid"),
    ("w4a4_route_experts_scored", dict(groups=3), "groups"),
    ("w4a4_route_experts_scored", dict(groups=2, top_groups=3), "top_groups"),
    ("w4a4_route_experts_scored", dict(groups=4, top_groups=1), "top_k"),
    ("w4a4_route_experts_scored", dict(top_k=5), "top_k"),
    ("w4a4_route_experts_scored", dict(top_k=0), "top_k"),
    ("w4a4_route_experts_scored", dict(group_best=3), "group_best"),
    ("w4a4_route_experts_scored", dict(bias=z(E, dtype=BF)), "bias"),
    ("w4a4_route_experts_scored", dict(bias=z(E + 1, dtype=F32)), "bias"),
    ("w4a4_route_experts_scored", dict(logits=z(E, M, dtype=BF).t()), "contiguous rows"),
    ("w8a8_experts_fp8", dict(w2_codes=z(E, K, 256), w2_scales=z(E, 3, 2, dtype=F32)), "must be"),
    ("w8a8_experts_fp8", dict(w13_codes=z(E, 224, K), w13_scales=z(E, 2, 3, dtype=F32), w2_codes=z(E, K, 112)), "F=112"),
    ("w8a8_experts_fp8", dict(logits=z(M, E + 1, dtype=BF)), "logits"),
    ("w8a8_experts_fp8", dict(rows_dtype=torch.float16), "rows_dtype"),
    ("w8a8_experts_fp8", dict(groups=4, top_groups=1, top_k=2), "top_k"),
]


@pytest.mark.parametrize("name,over,match", BAD, ids=[f"{i}-{n}" for i, (n, _, _) in enumerate(BAD)])
def test_binding_refuses(name, over, match):
    with pytest.raises(ValueError, match=match):
        getattr(b, name)(**args(name, **over))


@pytest.mark.parametrize("name", sorted({n for n, _, _ in BAD}))
def test_binding_refuses_the_cpu(name):
    with pytest.raises(ValueError, match="device"):
        getattr(b, name)(**args(name))


def test_float64_activations_are_not_implemented():
    for name, x in (("w8a8_quantize_fp8", "x"), ("w8a8_quantize_weights_fp8", "w"), ("w4a4_route_experts_scored", "logits")):
        shape = args(name)[x].shape
        with pytest.raises(NotImplementedError):
            getattr(b, name)(**args(name, **{x: torch.zeros(shape, dtype=torch.float64)}))


P = 0x1000   # an aligned pointer that nothing reads: every call ends in validation


def c(name, *a):
    return getattr(b.lib(), name)(*a)


def test_abi_refuses():
    I, U = b.INVALID, b.UNSUPPORTED
    quant = lambda **o: c("w8a8_quantize_fp8", *{**dict(x=P, dt=2, M=4, K=64, sm=64, sk=1, g=0, si=None, so=None, codes=P,  # noqa: E731
                                                         scales=P, st=None), **o}.values())
    assert quant(K=24, sm=24) == I and quant(M=-1) == I and quant(sm=-1) == I and quant(x=None) == I
    assert quant(codes=None) == I and quant(codes=P + 8) == U and quant(scales=P + 2) == U and quant(dt=9) == U
    assert quant(g=24) == U and quant(g=128) == I and quant(g=-1) == I and quant(g=64, si=P + 4) == U
    assert quant(K=1 << 23, sm=1 << 23) == U and quant(M=1 << 29) == U and quant(M=1 << 27, K=1024, sm=1024) == U
    wq = lambda **o: c("w8a8_quantize_weights_fp8", *{**dict(w=P, dt=2, E=2, N=4, K=64, se=256, sn=64, sk=1, g=0, si=None,  # noqa: E731
                                                              so=None, codes=P, scales=P, st=None), **o}.values())
    assert wq(E=-1) == I and wq(E=65536) == U and wq(K=40) == I and wq(se=-1) == I and wq(codes=None) == I
    gemm = lambda **o: c("w8a8_gemm_fp8", *{**dict(codes=P, scales=P, M=4, K=64, w=P, ws=P, N=16, bias=None, bdt=0, out=P,  # noqa: E731
                                                    odt=2, st=None), **o}.values())
    assert gemm(N=-1) == I and gemm(out=None) == I and gemm(odt=7) == U and gemm(bias=P, bdt=5) == U and gemm(w=None) == I
    assert gemm(codes=P + 4) == U and gemm(M=1 << 28, N=1 << 20) == U and gemm(M=1 << 27, K=1024) == U
    grp = lambda **o: c("w8a8_grouped_gemm_fp8", *{**dict(codes=P, scales=P, M=4, K=64, w=P, ws=P, E=2, N=16, off=P, rows=P,  # noqa: E731
                                                           R=8, bias=None, bdt=0, out=P, odt=2, st=None), **o}.values())
    assert grp(E=0) == I and grp(off=None) == I and grp(R=-1) == I and grp(rows=None) == I and grp(R=1 << 31) == U
    assert grp(E=20000) == U and grp(M=1 << 22, K=1024) == U and grp(N=1 << 22) == U and grp(N=1 << 21, odt=0) == U
    gat = lambda **o: c("w8a8_grouped_gated_fp8", *{**dict(codes=P, scales=P, M=4, K=64, w=P, ws=P, E=2, N=256, off=P, rows=P,  # noqa: E731
                                                            R=8, bias=None, bdt=0, oc=P, os=P, st=None), **o}.values())
    assert gat(N=128) == I and gat(oc=None) == I and gat(os=None) == I and gat(oc=P + 8) == U
    rt = lambda **o: c("w4a4_route_experts_scored", *{**dict(l=P, dt=2, T=4, s=8, E=8, k=2, sig=1, bias=None, groups=1, tg=1,  # noqa: E731
                                                              gb=1, rn=1, scale=1.0, w=P, e=P, rows=P, pos=P, off=P, ws=None,
                                                              wb=0, st=None), **o}.values())
    assert rt(groups=3) == I and rt(groups=0) == I and rt(groups=4, tg=5) == I and rt(groups=4, tg=0) == I and rt(gb=0) == I
    assert rt(groups=8, tg=1) == I and rt(E=2048, s=2048) == U and rt(E=1024, s=1024, groups=128, tg=64) == U
    assert rt(T=1 << 31) == U and rt(T=1000) == I and rt(off=None) == I and rt(s=4) == I and rt(k=9) == I
    big = 1 << 40
    ex = lambda **o: c("w8a8_experts_fp8", *{**dict(x=P, dt=2, T=4, K=64, sm=64, sk=1, g=0, si=None, so=None, l=P, ldt=2, ls=8,  # noqa: E731
                                                     E=8, k=2, sig=1, bias=None, groups=1, tg=1, gb=1, rn=1, scale=1.0, w13=P,
                                                     s13=P, F=128, w2=P, s2=P, rdt=2, out=P, ws=P, wb=big, st=None),
                                            **o}.values())
    assert ex(F=64) == I and ex(F=0) == I and ex(wb=16) == I and ex(ws=P + 8) == U and ex(out=None) == I and ex(rdt=1) == U
    assert ex(groups=3) == I and ex(k=9) == I and ex(T=1 << 27, k=2) == U and ex(T=-1) == I


def test_abi_exports_what_the_header_declares():
    src = re.sub(r"/\*.*?\*/", "", open(os.path.join(os.path.dirname(__file__), "..", "include", "w4a4.h")).read(), flags=re.S)
    names = set(re.findall(r"(w8a8_[a-z_0-9]*fp8[a-z_0-9]*)\s*\(", src))
    assert len(names) == 12 and names <= set(b._SIGNATURES)
    for n in names:
        assert hasattr(b.lib(), n)


def test_empty_calls_are_fine():
    assert c("w8a8_quantize_fp8", None, 2, 0, 64, 64, 1, 0, None, None, None, None, None) == b.OK
    assert c("w8a8_quantize_weights_fp8", None, 2, 0, 4, 64, 0, 64, 1, 0, None, None, None, None, None) == b.OK
    assert c("w8a8_gemm_fp8", None, None, 0, 64, P, P, 16, None, 0, None, 2, None) == b.OK
    assert b.w8a8_linear_fp8_workspace_size(0, 64) == 0 and b.w8a8_gemm_fp8_plan(0, 64, 64) == "none"
    assert b.w8a8_linear_fp8_workspace_size(5, 272) == 1536 + 256
    assert b.w8a8_experts_fp8_workspace_size(0, 64, 128, 8, 2, BF) == 0


def test_plain_codes_are_torchs():
    """The tests' grid and rounding against torch's own e4m3 conversion."""
    n = torch.arange(256, dtype=torch.uint8)
    v = n.view(F8).double().numpy()
    got = fp8.code_values(n.numpy())
    assert np.array_equal(np.isnan(v), np.isnan(got)) and np.array_equal(v[~np.isnan(v)], got[~np.isnan(v)])
    x = torch.randn(1 << 16, generator=torch.Generator().manual_seed(1)) * 100
    mid = torch.from_numpy((fp8.GRID[1:] + fp8.GRID[:-1]) / 2).float()   # ties
    x = torch.cat([x, mid, -mid]).clamp(-448, 448)
    want = x.to(F8).view(torch.uint8).numpy()
    assert np.array_equal(fp8.nearest_code(x.double().numpy()) | (np.signbit(x.numpy()) << 7), want)

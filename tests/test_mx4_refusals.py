"""CPU tests of the MX4 entry points: every wrong argument is refused before any device
access, by the binding (ValueError) and by the C ABI (status codes); host-only
queries; the scale layout's round trip."""
import ctypes
import os

import numpy as np
import pytest
import torch

from bit_quantized_linear_rotate_amd import _binding as b
from tests import mx4

pytestmark = pytest.mark.skipif(not os.path.exists(b.LIB_PATH), reason="libw4a4.so not built")

U8, BF, I32 = torch.uint8, torch.bfloat16, torch.int32
M, K, N, E = 6, 320, 48, 3


def z(*shape, dtype=U8):
    return torch.zeros(*shape, dtype=dtype)


def args(name, **over):
    """Well-formed CPU arguments: refused only for not being on a HIP device."""
    op = dict(codes=z(M, K // 2), scales=z(2, M, 8))
    w = dict(w_codes=z(N, K // 2), w_scales=z(2, N, 8))
    we = dict(w_codes=z(E, 64, K // 2), w_scales=z(E, 2, 64, 8))
    a = {
        "w4a4_quantize_mx4": dict(x=z(M, K, dtype=BF)),
        "w4a4_dequantize_mx4": dict(op),
        "w4a4_gemm_mx4": dict(op, **w),
        "w4a4_linear_mx4": dict(x=z(M, K, dtype=BF), **w),
        "w4a4_grouped_gemm_mx4": dict(op, **we, offsets=z(E + 1, dtype=I32)),
        "w4a4_grouped_gated_mx4": dict(op, **we, offsets=z(E + 1, dtype=I32)),
        "w4a4_route_experts": dict(logits=z(M, E, dtype=BF), top_k=2),
        "w4a4_combine_experts": dict(y=z(M, N, dtype=BF), pos=z(4, 2, dtype=I32), weights=torch.zeros(4, 2)),
        "w4a4_experts_mx4": dict(x=z(M, K, dtype=BF), logits=z(M, E, dtype=BF), top_k=2, w13_codes=z(E, 128, K // 2),
                                 w13_scales=z(E, 2, 128, 8), w2_codes=z(E, K, 32), w2_scales=z(E, 1, K, 8)),
    }[name]
    a.update(over)
    return a


BAD = [
    ("w4a4_quantize_mx4", dict(x=z(M, 40, dtype=BF)), "multiple of 32"),
    ("w4a4_quantize_mx4", dict(h=b.Hadamard(256)), "multiple of g"),
    ("w4a4_quantize_mx4", dict(h=torch.eye(64)), "Hadamard"),
    ("w4a4_dequantize_mx4", dict(scales=z(M, K // 32)), "scales"),
    ("w4a4_dequantize_mx4", dict(codes=z(M, K // 2 - 8)), "multiple of 32"),
    ("w4a4_dequantize_mx4", dict(codes=z(M, K // 2, dtype=torch.int8)), "codes"),
    ("w4a4_dequantize_mx4", dict(dtype=torch.int8), "dtype"),
    ("w4a4_gemm_mx4", dict(w_codes=z(N, K // 2 + 16), w_scales=z(2, N, 8)), "w_codes"),
    ("w4a4_gemm_mx4", dict(w_scales=z(1, N, 8)), "w_scales"),
    ("w4a4_gemm_mx4", dict(bias=z(N + 1, dtype=BF)), "bias"),
    ("w4a4_gemm_mx4", dict(out_dtype=torch.float64), "out_dtype"),
    ("w4a4_gemm_mx4", dict(codes=z(M, K)[:, ::2]), "contiguous"),
    ("w4a4_linear_mx4", dict(bias=z(N, dtype=torch.float32)), "bias"),
    ("w4a4_linear_mx4", dict(out=z(M, N + 1, dtype=BF)), "out"),
    ("w4a4_linear_mx4", dict(w_codes=z(N, 64), w_scales=z(1, N, 8)), "w_codes"),
    ("w4a4_grouped_gemm_mx4", dict(offsets=z(E, dtype=I32)), "offsets"),
    ("w4a4_grouped_gemm_mx4", dict(offsets=z(E + 1, dtype=torch.int64)), "offsets"),
    ("w4a4_grouped_gemm_mx4", dict(rows=z(M, dtype=torch.int64)), "rows"),
    ("w4a4_grouped_gemm_mx4", dict(rows=z(M, 1, dtype=I32)), "rows"),
    ("w4a4_grouped_gemm_mx4", dict(bias=z(E, 65, dtype=BF)), "bias"),
    ("w4a4_grouped_gemm_mx4", dict(w_scales=z(E, 64, 16)), "w_scales"),
    ("w4a4_grouped_gated_mx4", dict(w_codes=z(E, 96, K // 2), w_scales=z(E, 2, 96, 8)), "blocks of 32"),
    ("w4a4_route_experts", dict(top_k=0), "top_k"),
    ("w4a4_route_experts", dict(top_k=E + 1), "top_k"),
    ("w4a4_route_experts", dict(logits=z(M, 2 * E, dtype=BF)[:, ::2]), "contiguous rows"),
    ("w4a4_combine_experts", dict(weights=torch.zeros(4, 3)), "weights"),
    ("w4a4_combine_experts", dict(pos=z(4, dtype=I32)), "pos"),
    ("w4a4_combine_experts", dict(y=z(M, N)), "y"),
    ("w4a4_experts_mx4", dict(logits=z(M, E + 1, dtype=BF)), "logits"),
    ("w4a4_experts_mx4", dict(top_k=E + 1), "top_k"),
    ("w4a4_experts_mx4", dict(w2_codes=z(E, K, 48), w2_scales=z(E, 1, K, 8)), "w13_codes"),
    ("w4a4_experts_mx4", dict(out=z(M, K, dtype=torch.float32)), "out"),
]


@pytest.mark.parametrize("i", range(len(BAD)))
def test_binding_refuses(i):
    name, over, match = BAD[i]
    with pytest.raises(ValueError, match=match):
        getattr(b, name)(**args(name, **over))


@pytest.mark.parametrize("name", ["w4a4_quantize_mx4", "w4a4_dequantize_mx4", "w4a4_gemm_mx4", "w4a4_linear_mx4",
                                  "w4a4_grouped_gemm_mx4", "w4a4_grouped_gated_mx4", "w4a4_route_experts",
                                  "w4a4_combine_experts", "w4a4_experts_mx4"])
def test_host_tensors_are_refused(name):
    with pytest.raises(ValueError, match="CUDA"):
        getattr(b, name)(**args(name))


FAKE = ctypes.c_void_p(0x1000)   # never dereferenced: validation fails first


def test_abi_refusals():
    L = b.lib()
    q = lambda **o: L.w4a4_quantize_mx4(*{**dict(x=FAKE, dt=2, M=4, K=64, sm=64, sk=1, g=0, si=None, so=None, c=FAKE, s=FAKE,  # noqa: E731,E501
                                                 st=None), **o}.values())
    assert q(K=40) == b.INVALID and q(M=-1) == b.INVALID and q(x=None) == b.INVALID and q(c=None) == b.INVALID
    assert q(g=48) == b.UNSUPPORTED and q(g=128) == b.INVALID and q(g=-1) == b.INVALID and q(dt=5) == b.UNSUPPORTED
    assert q(c=ctypes.c_void_p(0x1008)) == b.UNSUPPORTED and q(K=0) == b.INVALID and q(M=0) == b.OK
    assert q(g=64, si=ctypes.c_void_p(0x1001)) == b.UNSUPPORTED and q(M=1 << 29) == b.UNSUPPORTED
    g = lambda **o: L.w4a4_gemm_mx4(*{**dict(a=FAKE, sa=FAKE, M=4, K=64, w=FAKE, sw=FAKE, N=8, b=None, bd=0, o=FAKE, od=2,  # noqa: E731,E501
                                             st=None), **o}.values())
    assert g(K=33) == b.INVALID and g(a=None) == b.INVALID and g(sw=None) == b.INVALID and g(o=None) == b.INVALID
    assert g(od=9) == b.UNSUPPORTED and g(b=FAKE, bd=9) == b.UNSUPPORTED and g(N=-1) == b.INVALID
    assert g(M=1 << 28, N=1 << 20) == b.UNSUPPORTED and g(M=0) == b.OK and g(N=0) == b.OK
    gg = lambda **o: L.w4a4_grouped_gemm_mx4(*{**dict(a=FAKE, sa=FAKE, M=4, K=64, w=FAKE, sw=FAKE, E=2, N=8, off=FAKE,  # noqa: E731,E501
                                                      rows=FAKE, R=4, b=None, bd=0, o=FAKE, od=2, st=None), **o}.values())
    assert gg(E=0) == b.INVALID and gg(R=-1) == b.INVALID and gg(off=None) == b.INVALID and gg(rows=None, R=5) == b.INVALID
    assert gg(R=1 << 31) == b.UNSUPPORTED and gg(M=1 << 27) == b.UNSUPPORTED and gg(R=0) == b.OK
    gt = lambda **o: L.w4a4_grouped_gated_mx4(*{**dict(a=FAKE, sa=FAKE, M=4, K=64, w=FAKE, sw=FAKE, E=2, N=64, off=FAKE,  # noqa: E731,E501
                                                       rows=FAKE, R=4, b=None, bd=0, oc=FAKE, os=FAKE, st=None), **o}.values())
    assert gt(N=96) == b.INVALID and gt(oc=None) == b.INVALID and gt(os=None) == b.INVALID
    assert gt(oc=ctypes.c_void_p(0x1004)) == b.UNSUPPORTED and gt(R=0) == b.OK
    r = lambda **o: L.w4a4_route_experts(*{**dict(l=FAKE, dt=0, T=4, s=8, E=8, k=2, n=1, w=FAKE, e=FAKE, r=FAKE, p=FAKE,  # noqa: E731,E501
                                                  o=FAKE, ws=None, b=0, st=None), **o}.values())
    assert r(k=9) == b.INVALID and r(k=0) == b.INVALID and r(s=7) == b.INVALID and r(E=2000, s=2000) == b.UNSUPPORTED
    assert r(k=33, E=40, s=40) == b.UNSUPPORTED and r(T=1000) == b.INVALID and r(o=None) == b.INVALID and r(dt=4) == b.UNSUPPORTED
    assert b"workspace" in L.w4a4_last_error() or r(T=1000) == b.INVALID
    c = lambda **o: L.w4a4_combine_experts(*{**dict(y=FAKE, dt=0, R=4, N=8, p=FAKE, w=FAKE, T=4, k=2, o=FAKE, st=None),  # noqa: E731,E501
                                             **o}.values())
    assert c(k=0) == b.INVALID and c(y=None) == b.INVALID and c(N=-1) == b.INVALID and c(dt=7) == b.UNSUPPORTED and c(T=0) == b.OK


def test_linear_and_experts_refuse_small_workspaces():
    L = b.lib()
    need = b.w4a4_linear_mx4_workspace_size(M, K)
    assert need >= M * K // 2 + 2 * M * 8
    rc = L.w4a4_linear_mx4(FAKE, 2, M, K, K, 1, 0, None, None, FAKE, FAKE, N, None, FAKE, 2, FAKE, need - 1, None)
    assert rc == b.INVALID and b"workspace" in L.w4a4_last_error()
    need = b.w4a4_experts_mx4_workspace_size(M, K, 64, E, 2, BF)
    assert need > 0 and b.w4a4_experts_mx4_workspace_size(0, K, 64, E, 2, BF) == 0
    rc = L.w4a4_experts_mx4(FAKE, 2, M, K, K, 1, 0, None, None, FAKE, 0, E, E, 2, 1, FAKE, FAKE, 64, FAKE, FAKE, FAKE,
                            FAKE, need - 1, None)
    assert rc == b.INVALID and b"workspace" in L.w4a4_last_error()


def test_scale_layout_round_trip():
    r = np.random.default_rng(0)
    for lead, rows, k in (((), 5, 320), ((2,), 7, 256), ((), 1, 32), ((3,), 4, 1312)):
        s = r.integers(0, 255, (*lead, rows, k // 32)).astype(np.uint8)
        t = b.mx4_scales_from_rows(torch.from_numpy(s))
        assert np.array_equal(t.numpy(), mx4.slabs(s)) and t.is_contiguous()
        assert np.array_equal(b.mx4_scales_to_rows(t, k).numpy(), s)
        assert np.array_equal(mx4.unslab(t.numpy(), k), s)


def test_oracle_quantizer_on_hand_computed_blocks():
    y = np.zeros((3, 32))
    y[0, :9] = [6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -0.24]      # X = 0: ties to even
    y[1, 0], y[1, 1] = 7.9, -1.0                                    # saturates at 6
    y[2, 0], y[2, 1] = 8.0, 1.0                                     # X = 1
    c, s = mx4.quantize(y)
    n = np.stack([c & 15, c >> 4], -1).reshape(3, 32)
    assert list(s[:, 0]) == [127, 127, 128]
    assert list(n[0, :9]) == [7, 6, 6, 4, 4, 2, 2, 0, 8] and list(n[1, :2]) == [7, 10] and list(n[2, :2]) == [6, 1]
    assert mx4.scale_exponent(0.0) == -127 and mx4.scale_exponent(2.0 ** -140) == -127


def test_plan_names():
    assert b.w4a4_gemm_mx4_plan(1, 3840, 3840) == "skinny"
    assert b.w4a4_gemm_mx4_plan(8192, 3840, 3840) == "tile256"
    assert b.w4a4_gemm_mx4_plan(0, 256, 64) == "none"
    with pytest.raises(ValueError):
        b.w4a4_gemm_mx4_plan(4, 40, 64)

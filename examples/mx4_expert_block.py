"""A feed-forward block of experts on MX4, as a model would hold it.

The weights are quantized once, rotated like the activations that will meet
them: y = x R, so (x R)(w R)^T = x w^T.  A call routes its tokens, runs the
expert layer and adds a projection that every token takes.

    python examples/mx4_expert_block.py [--tokens 4096]

prints how far the block is from single precision and how long a call takes.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_quantized_linear_rotate_amd as w4  # noqa: E402


class ExpertBlock:
    """w13 (E, 2 F, K): gates, then ups; w2 (E, K, F); router (E, K); shared (K, K)."""

    def __init__(self, w13, w2, router, shared, top_k, group=64):
        self.h, self.top_k, self.router = w4.Hadamard(group), top_k, router
        self.w13 = self.experts(w13, self.h)
        self.w2 = self.experts(w2, None)          # meets the gated results, which are not rotated
        self.shared = w4.w4a4_quantize_mx4(shared, self.h)

    @staticmethod
    def experts(w, h):
        codes, scales = zip(*(w4.w4a4_quantize_mx4(e, h) for e in w))
        return torch.stack(codes), torch.stack(scales)

    def __call__(self, x):
        logits = x @ self.router.t()
        y = w4.w4a4_experts_mx4(x, logits, self.top_k, *self.w13, *self.w2, h=self.h)
        return y + w4.w4a4_linear_mx4(x, *self.shared, h=self.h)


def plain(x, w13, w2, router, shared, top_k):
    """The same block in single precision."""
    x, w13, w2, shared = x.float(), w13.float(), w2.float(), shared.float()
    weights, experts = torch.topk(x @ router.float().t(), top_k, dim=-1)
    weights = torch.softmax(weights, -1)
    out = x @ shared.t()
    for e in range(w13.shape[0]):
        t, j = torch.where(experts == e)
        gate, up = (x[t] @ w13[e].t()).chunk(2, -1)
        out.index_add_(0, t, weights[t, j, None] * ((torch.nn.functional.silu(gate) * up) @ w2[e].t()))
    return out


def main(tokens=4096, K=3840, F=1280, E=32, top_k=4, repeat=20):
    torch.manual_seed(0)
    d = dict(device="cuda", dtype=torch.bfloat16)
    w13, w2 = torch.randn(E, 2 * F, K, **d) * K ** -0.5, torch.randn(E, K, F, **d) * F ** -0.5
    router, shared = torch.randn(E, K, **d) * K ** -0.5, torch.randn(K, K, **d) * K ** -0.5
    x = torch.randn(tokens, K, **d)
    block = ExpertBlock(w13, w2, router, shared, top_k)
    want = plain(x, w13, w2, router, shared, top_k)
    off = float((block(x).float() - want).norm() / want.norm())
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(repeat):
        block(x)
    end.record()
    torch.cuda.synchronize()
    us = start.elapsed_time(end) / repeat * 1e3
    print(f"{tokens} tokens, {E} experts of {K} x {F}, {top_k} each: {off:.3f} off single precision, {us:.0f} us a call")
    return off


if __name__ == "__main__":
    p = argparse.ArgumentParser()
    p.add_argument("--tokens", type=int, default=4096)
    main(p.parse_args().tokens)

"""The mixture-of-experts half of a decoder layer, activations MXFP8 between its kernels:

    h = h + attention output; y = RMSNorm(h), as bf16 for the gate and MXFP8 for the experts
    gate logits -> 8 of 64 experts and their weights per token
    out = the experts' products, added to the stream by the next layer's first call

``python examples/moe_half_layer.py [--tokens T]`` builds random weights, captures the half-layer in a
CUDA graph and prints its time per step.
"""
from __future__ import annotations

import argparse
import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mxfp8_activation_quant_gb300 as mxq  # noqa: E402


@dataclass
class Weights:
    gamma: torch.Tensor   # bf16 [H]
    gate: torch.Tensor    # bf16 [E, H]
    bias: torch.Tensor    # fp32 [E], the balance bias of the router
    w13: mxq.MXFP8        # [E * 2 I, H], rows alternate gate, up
    w2: mxq.MXFP8         # [E * H, I]

    @staticmethod
    def random(E: int, H: int, I: int, seed: int = 0) -> "Weights":
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, std=1.0):
            return (torch.randn(shape, generator=g, device="cuda") * std).to(torch.bfloat16)

        def quantized(w):
            q, sf = mxq.quantize(w, layouts=(mxq.SF_TILED_128X4,))
            return mxq.MXFP8(q, sf[mxq.SF_TILED_128X4])

        return Weights(gamma=(1.0 + 0.1 * normal(H).float()).to(torch.bfloat16), gate=normal(E, H, std=H ** -0.5),
                       bias=0.05 * normal(E).float(),
                       w13=quantized(mxq.interleave_gate_up(normal(E, I, H, std=H ** -0.5), normal(E, I, H, std=H ** -0.5))),
                       w2=quantized(normal(E * H, I, std=I ** -0.5)))


class HalfLayer:
    """Buffers of one batch size; step() enqueues the half-layer on the current stream."""

    def __init__(self, w: Weights, T: int, k: int = 8, groups: int = 8, topk_groups: int = 4, eps: float = 1e-6):
        (E, H), dev = w.gate.shape, w.gate.device
        I = w.w2.data.shape[1]
        self.w, self.groups, self.topk_groups, self.eps = w, groups, topk_groups, eps
        self.y = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
        self.yq = torch.empty((T, H), dtype=torch.uint8, device=dev)
        self.ysf = mxq.empty_sf(mxq.SF_ROWMAJOR_U8, T, H, dev)
        self.logits = torch.empty((T, E), dtype=torch.bfloat16, device=dev)
        self.ids = torch.empty((T, k), dtype=torch.int32, device=dev)
        self.weights = torch.empty((T, k), dtype=torch.float32, device=dev)
        self.out = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
        self.workspace = torch.empty(mxq.moe_workspace_bytes(T, k, E, H, I), dtype=torch.uint8, device=dev)
        self.status = mxq.new_status(dev)

    def step(self, x: torch.Tensor, h: torch.Tensor) -> torch.Tensor:
        """x: bf16 [T, H], the attention's output; h: the residual stream, updated in place. Returns the
        experts' output, the `x` of the next half-layer."""
        w = self.w
        mxq.add_rmsnorm_dual_out(x, h, w.gamma, self.eps, h, self.y, self.yq, sf_rowmajor=self.ysf)
        torch.matmul(self.y, w.gate.t(), out=self.logits)
        mxq.moe_route(self.logits, self.ids, self.weights, bias=w.bias, groups=self.groups, topk_groups=self.topk_groups,
                      scale=2.5)
        mxq.moe_experts_mxfp8(mxq.MXFP8(self.yq, self.ysf, mxq.SF_ROWMAJOR_U8), self.ids, self.weights, w.w13, w.w2,
                              self.out, status=self.status, workspace=self.workspace)
        return self.out


def main() -> None:
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--tokens", type=int, default=64)
    p.add_argument("--experts", type=int, default=64)
    p.add_argument("--hidden", type=int, default=5120)
    p.add_argument("--intermediate", type=int, default=1024)
    a = p.parse_args()
    layer = HalfLayer(Weights.random(a.experts, a.hidden, a.intermediate), a.tokens)
    x = torch.randn((a.tokens, a.hidden), device="cuda").to(torch.bfloat16)
    h = torch.randn((a.tokens, a.hidden), device="cuda").to(torch.bfloat16)
    layer.step(x, h)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.step(x, h)
    for _ in range(5):
        graph.replay()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    n = 50
    start.record()
    for _ in range(n):
        graph.replay()
    end.record()
    end.synchronize()
    mxq.check_status(layer.status)
    print(f"{a.tokens} tokens, {a.experts} experts, {a.hidden} -> 2 x {a.intermediate}: "
          f"{1e3 * start.elapsed_time(end) / n:.1f} us per half-layer")


if __name__ == "__main__":
    main()

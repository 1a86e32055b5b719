"""The attention of a decode step over a paged latent cache, MXFP8 from the cache to the output projection:

    this step's tokens into their slots of the cache (MXFP8)
    o = attention of 64 heads of 512 over each sequence, as the MXFP8 operand of
    out = _o_proj(o)

``python examples/attention_half_layer.py [--sequences B] [--tokens N]`` fills a cache with N random tokens a
sequence, captures a step in a CUDA graph and prints its time.
"""
from __future__ import annotations

import argparse
import os
import sys
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mxfp8_activation_quant_gb300 as mxq  # noqa: E402
from mxfp8_activation_quant_gb300 import synth  # noqa: E402

HEADS, DIM, PAGE = 64, 512, 64


@dataclass
class Weights:
    wa: mxq.MXFP8   # [G * Na, Ka]
    wb: mxq.MXFP8   # [Nb, G * Na]

    @staticmethod
    def random(seed: int = 0) -> "Weights":
        def quantized(w):
            q, sf = mxq.quantize(w.cuda(), layouts=(mxq.SF_TILED_128X4,))
            return mxq.MXFP8(q, sf[mxq.SF_TILED_128X4])

        return Weights(wa=quantized(synth.wo_a_weight(seed, device="cuda")), wb=quantized(synth.wo_b_weight(seed, device="cuda")))


class HalfLayer:
    """A cache of `pages` pages, a table of `width` of them for each of B sequences, and a step's buffers."""

    def __init__(self, w: Weights, B: int, pages: int, width: int, scale: float = DIM ** -0.5):
        self.w, self.B, self.scale = w, B, scale
        self.cache = mxq.MXFP8Cache.empty(pages, PAGE, 1, DIM)
        self.table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
        self.o = torch.empty((B, HEADS * DIM), dtype=torch.uint8, device="cuda")
        self.osf = mxq.empty_sf(mxq.SF_TILED_128X4, B, HEADS * DIM)
        self.z = torch.empty((B, synth.KB), dtype=torch.uint8, device="cuda")
        self.zsf = mxq.empty_sf(mxq.SF_TILED_128X4, B, synth.KB)
        self.out = torch.empty((B, synth.NB), dtype=torch.bfloat16, device="cuda")
        self.workspace = torch.empty(mxq.paged_attention_workspace_bytes(B, HEADS, 1, DIM), dtype=torch.uint8, device="cuda")
        self.status = mxq.new_status()

    def prefill(self, kv: torch.Tensor, slots: torch.Tensor) -> None:
        """kv: bf16 [T, 512], a prompt's latent rows, into their slots."""
        mxq.kv_write_mxfp8(kv.unsqueeze(1), slots, self.cache)

    def step(self, q: torch.Tensor, kv: torch.Tensor, slots: torch.Tensor, seq_lens: torch.Tensor) -> torch.Tensor:
        """q: bf16 [B, 64, 512]; kv: bf16 [B, 512], this step's rows, and their slots int32 [B]; seq_lens int32 [B],
        with this step's token. Returns the layer's output, bf16 [B, 5120]."""
        mxq.kv_write_mxfp8(kv.unsqueeze(1), slots, self.cache)
        mxq.paged_attention_mxfp8(q, self.cache, self.table, seq_lens, self.scale, out_q=self.o, sf_128x4=self.osf,
                                  status=self.status, workspace=self.workspace)
        mxq.o_proj_mxfp8(mxq.MXFP8(self.o, self.osf), self.w.wa, self.w.wb, self.B, synth.G, synth.NA, synth.KA, synth.NB,
                         self.z, self.zsf, self.out, status=self.status)
        return self.out


def main() -> None:
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    p.add_argument("--sequences", type=int, default=32)
    p.add_argument("--tokens", type=int, default=4096)
    a = p.parse_args()
    B, n = a.sequences, a.tokens
    width = -(-(n + 1) // PAGE)
    layer = HalfLayer(Weights.random(), B, B * width, width)
    layer.table.copy_(torch.randperm(B * width, device="cuda").view(B, width))
    positions = torch.arange(n, device="cuda")
    for b in range(B):
        layer.prefill(torch.randn((n, DIM), device="cuda").to(torch.bfloat16),
                      layer.table[b, positions // PAGE] * PAGE + (positions % PAGE).int())
    q = torch.randn((B, HEADS, DIM), device="cuda").to(torch.bfloat16)
    kv = torch.randn((B, DIM), device="cuda").to(torch.bfloat16)
    slots = layer.table[:, n // PAGE] * PAGE + n % PAGE
    lens = torch.full((B,), n + 1, dtype=torch.int32, device="cuda")
    layer.step(q, kv, slots, lens)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.step(q, kv, slots, lens)
    for _ in range(5):
        graph.replay()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    steps = 50
    start.record()
    for _ in range(steps):
        graph.replay()
    end.record()
    end.synchronize()
    mxq.check_status(layer.status)
    print(f"{B} sequences of {n} tokens, {HEADS} heads of {DIM}: {1e3 * start.elapsed_time(end) / steps:.1f} us per step")


if __name__ == "__main__":
    main()

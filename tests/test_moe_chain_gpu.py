"""The three mixture-of-experts operators together (examples/moe_half_layer.py): each stage against its
definition on the stage before it, and the captured half-layer against the eager one."""
import importlib.util
import os

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    from mxfp8_activation_quant_gb300 import build

    build.build()
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    spec = importlib.util.spec_from_file_location("moe_half_layer", os.path.join(ROOT, "examples", "moe_half_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def values(q, sf):
    scale = ((sf.long() + 896) << 52).view(torch.float64)
    return q.view(torch.float8_e4m3fn).double() * scale.view(q.shape[0], -1).repeat_interleave(32, dim=1)


def untile(sf, rows, cols):
    """F8_128x4 scales -> row-major [rows, cols / 32]."""
    return sf.view(rows // 128, cols // 128, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rows, cols // 32)


@pytest.mark.parametrize("T", [1, 5, 130])
def test_half_layer(example, T):
    E, H, I, k = 64, 512, 256, 8
    w = example.Weights.random(E, H, I)
    layer = example.HalfLayer(w, T, k)
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    h0 = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16)
    h = h0.clone()
    out = layer.step(x, h)
    example.mxq.check_status(layer.status)
    assert torch.equal(h, (x.float() + h0.float()).to(torch.bfloat16))
    # the router on the gate's logits: every token's experts by the definition
    s = torch.sigmoid(layer.logits.double())
    c = s + w.bias.double()
    for t in range(T):
        groups = c[t].view(8, 8).topk(2, dim=1).values.sum(1).topk(4).indices
        left = torch.full_like(c[t], -1e9).view(8, 8)
        left[groups] = c[t].view(8, 8)[groups]
        top = left.view(-1).topk(k).indices
        assert set(top.tolist()) == set(layer.ids[t].tolist())
        np.testing.assert_allclose(layer.weights[t].double().cpu(),
                                   (2.5 * s[t][layer.ids[t].long()] / s[t][top].sum()).cpu(), rtol=2.0 ** -18)
    # the experts on the norm's MXFP8 output
    yv = values(layer.yq, layer.ysf)
    w13 = values(w.w13.data, untile(w.w13.sf, E * 2 * I, H))
    w2 = values(w.w2.data, untile(w.w2.sf, E * H, I))
    ref = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    for t in range(T):
        for j in range(k):
            e = int(layer.ids[t, j])
            gu = w13[e * 2 * I:(e + 1) * 2 * I] @ yv[t]
            a = (gu[0::2] * torch.sigmoid(gu[0::2]) * gu[1::2]).to(torch.bfloat16)[None]
            q, sf = example.mxq.quantize(a, layouts=(0,))
            ref[t] += layer.weights[t, j].double() * (w2[e * H:(e + 1) * H] @ values(q, sf[0])[0])
    # two bf16 roundings and a few activations on the other side of a rounding, as in the experts' test
    assert ((out.double() - ref).norm() / ref.norm()).item() <= 4e-3


def test_captured_half_layer(example):
    T = 24
    w = example.Weights.random(64, 512, 256, seed=1)
    layer = example.HalfLayer(w, T)
    x = torch.randn((T, 512), device="cuda").to(torch.bfloat16)
    h0 = torch.randn((T, 512), device="cuda").to(torch.bfloat16)
    h = h0.clone()
    want = layer.step(x, h).clone()
    want_h = h.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        layer.step(x, h)
    for _ in range(2):
        h.copy_(h0)
        layer.out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(layer.out, want) and torch.equal(h, want_h)

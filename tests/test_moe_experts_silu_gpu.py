"""silu far below zero in moe_experts_mxfp8: g e^g is small, not zero, and a large u brings it back."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mxq():
    from mxfp8_activation_quant_gb300 import build

    build.build()
    import mxfp8_activation_quant_gb300 as m

    assert torch.cuda.is_available(), "GPU tests need CUDA"
    m.load()
    return m


@pytest.mark.parametrize("T", [1, 40, 400])  # (400 tokens of one expert: rows copied)
def test_large_negative_gates(mxq, T):
    """One group of 32 features for each gate value, u = 2^100 in all, W2 the identity."""
    H = I = 128
    gates = torch.tensor([-72.0, -88.0, -96.0, -104.0], device="cuda").repeat_interleave(32)
    wg = torch.zeros((1, I, H), device="cuda")
    wu = torch.zeros_like(wg)
    wg[0, :, 0] = gates
    wu[0, :, 1] = 2.0 ** 100
    x = torch.zeros((T, H), device="cuda")
    x[:, :2] = 1.0
    x[1::3, 0] = -0.5  # 36 .. 52: g itself
    mx = lambda t: mxq.MXFP8(*(lambda r: (r[0], r[1][2]))(  # noqa: E731
        mxq.quantize(t.to(torch.bfloat16).contiguous(), layouts=(2,))))
    w13 = mx(mxq.interleave_gate_up(wg, wu))
    w2 = mx(torch.eye(H, I, device="cuda"))
    out = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    ids = torch.zeros((T, 1), dtype=torch.int32, device="cuda")
    mxq.moe_experts_mxfp8(mx(x), ids, torch.ones((T, 1), device="cuda"), w13, w2, out)
    g = x[:, :1].double() * gates.double()
    want = g / (1.0 + torch.exp(-g)) * 2.0 ** 100
    # roundings to bf16 (the activation and the output, 2^-8 each) and to E4M3 (2^-4), fp32 before
    assert ((out.double() - want).abs() <= (2.0 ** -4 + 2.0 ** -7 + 2.0 ** -10) * want.abs()).all()

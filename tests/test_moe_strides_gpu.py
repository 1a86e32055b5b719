"""The mixture-of-experts calls on rows whose strides are unusual: a single row, whose stride means
nothing, and rows more than 2^31 elements apart."""
import pytest
import torch

pytestmark = pytest.mark.gpu
FAR = 2 ** 31 + 128


@pytest.fixture(scope="module")
def mxq():
    from mxfp8_activation_quant_gb300 import build

    build.build()
    import mxfp8_activation_quant_gb300 as m

    assert torch.cuda.is_available(), "GPU tests need CUDA"
    m.load()
    return m


def strided(t, stride):
    """t's rows, `stride` elements apart."""
    T, n = t.shape
    s = torch.empty((T - 1) * stride + n if T > 1 else n, dtype=t.dtype, device="cuda").as_strided((T, n), (stride, 1))
    s.copy_(t)
    return s


@pytest.mark.parametrize("T,stride", [(1, 1), (1, 5), (1, 2 ** 41), (2, FAR)])
def test_strides(mxq, T, stride):
    E, H, I, k = 8, 256, 128, 2
    g = torch.Generator(device="cuda").manual_seed(T)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    x, r, gamma = rnd(T, H), rnd(T, H), rnd(H)
    h, y, yq, sf = torch.empty_like(r), torch.empty_like(x), torch.empty((T, H), dtype=torch.uint8, device="cuda"), mxq.empty_sf(0, T, H)
    mxq.add_rmsnorm_dual_out(x, r, gamma, 1e-6, h, y, yq, sf_rowmajor=sf)
    y2, r2 = torch.empty_like(y), strided(r, stride)
    mxq.add_rmsnorm_dual_out(strided(x, stride), r2, gamma, 1e-6, r2, y2)
    assert torch.equal(y, y2) and torch.equal(h, r2)
    del r2

    logits = torch.randn((T, E), generator=g, device="cuda")
    ids, w = torch.empty((T, k), dtype=torch.int32, device="cuda"), torch.empty((T, k), device="cuda")
    mxq.moe_route(logits, ids, w)
    ids2, w2 = torch.empty_like(ids), torch.empty_like(w)
    mxq.moe_route(strided(logits, stride), ids2, w2)
    assert torch.equal(ids, ids2) and torch.equal(w, w2)

    mx = lambda t: mxq.MXFP8(*(lambda q: (q[0], q[1][2]))(mxq.quantize(t.contiguous(), layouts=(2,))))  # noqa: E731
    w13, wd = mx(rnd(E * 2 * I, H)), mx(rnd(E * H, I))
    out = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    mxq.moe_experts_mxfp8(mxq.MXFP8(yq, sf, 0), ids, w, w13, wd, out)
    out2 = strided(torch.zeros_like(out), stride)
    mxq.moe_experts_mxfp8(mxq.MXFP8(strided(yq, stride), sf, 0), ids, w, w13, wd, out2)
    assert torch.equal(out, out2)

"""add_rmsnorm_dual_out on the GPU: the residual stream exactly, bf16 y against the formula in 64
bits, and the MXFP8 y bit-identical to the standalone quantizer on the GPU's own y."""
import numpy as np
import pytest
import torch

from helpers import Guarded, bf16_ulp

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mxq():
    from mxfp8_activation_quant_gb300 import build

    build.build()
    import mxfp8_activation_quant_gb300 as m

    assert torch.cuda.is_available(), "GPU tests need CUDA"
    m.load()
    return m


def inputs(T, H, dtype, seed=0, pad_x=0, pad_r=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((T, H + pad_x), generator=g, device="cuda").to(torch.bfloat16)[:, :H]
    r = (3.0 * torch.randn((T, H + pad_r), generator=g, device="cuda"))
    r[:, 5 % H] *= 40.0
    r = r.to(dtype)[:, :H]
    gamma = (1.0 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(torch.bfloat16)
    return x, r, gamma


def check(mxq, x, r, gamma, eps, h, y, yq, pk, rm, tl):
    T, H = x.shape
    # fp32 sums of two bf16 or fp32 values, rounded once
    want_h = (x.float() + r.float()).to(r.dtype)
    assert torch.equal(h, want_h)
    # y is the exact value rounded to fp32 and then to bf16: half an ulp of each
    hd = h.double().cpu().numpy()
    ref = hd / np.sqrt((hd * hd).mean(1, keepdims=True) + eps) * gamma.double().cpu().numpy()
    if y is not None:
        assert (np.abs(y.double().cpu().numpy() - ref) / bf16_ulp(ref)).max() <= 0.5 + 2.0 ** -16
    if yq is not None:
        src = y if y is not None else torch.from_numpy(ref).cuda().float().to(torch.bfloat16)
        q2 = torch.empty((T, H), dtype=torch.uint8, device="cuda")
        rm2, tl2 = mxq.empty_sf(0, T, H), mxq.empty_sf(2, T, H)
        pk2 = mxq.empty_sf(1, T, H) if H % 128 == 0 else None
        mxq.mxfp8_quantize(src, q2, rm2, pk2, tl2)
        if y is not None:
            assert torch.equal(q2, yq)
            assert rm is None or torch.equal(rm2, rm)
            assert pk is None or torch.equal(pk2, pk)
            assert tl is None or torch.equal(tl2, tl)
        else:  # the GPU's own y is not there: all but a few elements next to a rounding border agree
            assert (q2 == yq).float().mean() > 0.995


SHAPES = [(1, 5120), (1, 32), (3, 96), (7, 5120), (129, 1056), (300, 7168), (513, 2080), (600, 16384), (2, 16384), (2050, 640), (600, 512),
          (513, 1056), (700, 5120), (530, 10240), (513, 7680)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", SHAPES)
def test_all_outputs(mxq, T, H, dtype):
    x, r, gamma = inputs(T, H, dtype)
    h = Guarded(T * H * r.element_size())
    y, yq, rm, tl = Guarded(T * H * 2), Guarded(T * H), Guarded(mxq.sf_bytes(0, T, H)), Guarded(mxq.sf_bytes(2, T, H))
    pk = Guarded(mxq.sf_bytes(1, T, H)) if H % 128 == 0 else None
    hv, yv, qv = h.view(dtype, (T, H)), y.view(torch.bfloat16, (T, H)), yq.view(shape=(T, H))
    mxq.add_rmsnorm_dual_out(x, r, gamma, 1e-6, hv, yv, qv, pk.body if pk else None, rm.body, tl.body)
    torch.cuda.synchronize()
    assert all(g.intact() for g in (h, y, yq, rm, tl)) and (pk is None or pk.intact())
    check(mxq, x, r, gamma, 1e-6, hv, yv, qv, pk.body if pk else None, rm.body, tl.body)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", [(1, 5120), (65, 2080)])
def test_in_place_strided_and_partial_outputs(mxq, T, H, dtype):
    x, r, gamma = inputs(T, H, dtype, 1, pad_x=24, pad_r=40)
    want = r.clone()
    y = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    mxq.add_rmsnorm_dual_out(x, r, gamma, 1e-5, r, y)  # bf16 only, in place
    check(mxq, x, want, gamma, 1e-5, r, y, None, None, None, None)
    # MXFP8 only
    r2 = want.clone()
    yq, rm = torch.empty((T, H), dtype=torch.uint8, device="cuda"), mxq.empty_sf(0, T, H)
    mxq.add_rmsnorm_dual_out(x, want, gamma, 1e-5, r2, yq=yq, sf_rowmajor=rm)
    check(mxq, x, want, gamma, 1e-5, r2, None, yq, None, rm, None)
    q2, s2 = mxq.quantize(y, layouts=(0,))
    assert torch.equal(q2, yq) and torch.equal(s2[0], rm)


def test_equals_rmsnorm_of_the_stored_stream(mxq):
    """The norm reads the stored stream: within the roundings of two sums in different orders it is
    rmsnorm_dual_out of residual_out."""
    T, H = 64, 5120
    x, r, gamma = inputs(T, H, torch.bfloat16, 2)
    h, y = torch.empty_like(r), torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    mxq.add_rmsnorm_dual_out(x, r, gamma, 1e-6, h, y)
    y2, q2 = torch.empty_like(y), torch.empty((T, H), dtype=torch.uint8, device="cuda")
    mxq.rmsnorm_dual_out(h, gamma, 1e-6, y2, q2, sf_rowmajor=mxq.empty_sf(0, T, H))
    d = (y.float() - y2.float()).abs().cpu().numpy()
    assert (d / bf16_ulp(y2.float().cpu().numpy())).max() <= 1.0 and (d > 0).mean() < 0.01


def test_zero_and_constant_rows(mxq):
    T, H = 3, 512
    x = torch.zeros((T, H), dtype=torch.bfloat16, device="cuda")
    r = torch.zeros_like(x)
    x[1] = 2.0
    r[1] = 1.0
    x[2], r[2] = 5.0, -5.0  # cancels exactly
    gamma = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    h, y = torch.empty_like(r), torch.empty_like(x)
    yq, rm = torch.empty((T, H), dtype=torch.uint8, device="cuda"), mxq.empty_sf(0, T, H)
    mxq.add_rmsnorm_dual_out(x, r, gamma, 1e-6, h, y, yq, sf_rowmajor=rm)
    assert torch.all(h[0] == 0) and torch.all(h[1] == 3) and torch.all(h[2] == 0)
    assert torch.all(y[0] == 0) and torch.all(y[2] == 0) and torch.all(y[1] == 1)
    assert torch.all(yq[0] == 0) and torch.all(rm.view(T, -1)[0] == 0) and torch.all(rm.view(T, -1)[2] == 0)


def test_offsets_past_32_bits(mxq):
    """2^31 elements and a few rows more, in place: sampled rows against the same rows alone."""
    H = 16384
    T = 2 ** 31 // H + 5
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn((T, H), generator=g, device="cuda", dtype=torch.bfloat16)
    r = torch.randn((T, H), generator=g, device="cuda", dtype=torch.bfloat16)
    gamma = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    t = torch.tensor([0, 1, 70000, T - 6, T - 2, T - 1], device="cuda")
    x1, r1 = x[t].contiguous(), r[t].contiguous()
    yq, tl = torch.empty((T, H), dtype=torch.uint8, device="cuda"), mxq.empty_sf(2, T, H)
    mxq.add_rmsnorm_dual_out(x, r, gamma, 1e-6, r, yq=yq, sf_128x4=tl)
    yq1, rm1 = torch.empty((6, H), dtype=torch.uint8, device="cuda"), mxq.empty_sf(0, 6, H)
    mxq.add_rmsnorm_dual_out(x1, r1, gamma, 1e-6, r1, yq=yq1, sf_rowmajor=rm1)
    assert torch.equal(r[t], r1) and torch.equal(yq[t], yq1)
    # the tiled scales of those rows
    c = torch.arange(H // 32, device="cuda")
    at = ((t[:, None] // 128) * (H // 128) + c // 4) * 512 + (t[:, None] % 32) * 16 + (t[:, None] % 128) // 32 * 4 + c % 4
    assert torch.equal(tl[at.reshape(-1)], rm1)


def test_other_stream_and_graph(mxq):
    T, H = 33, 1024
    x, r, gamma = inputs(T, H, torch.bfloat16, 3)
    h, y = torch.empty_like(r), torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    mxq.add_rmsnorm_dual_out(x, r, gamma, 1e-6, h, y, stream=s)
    s.synchronize()
    want = (h.clone(), y.clone())
    h.zero_(), y.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mxq.add_rmsnorm_dual_out(x, r, gamma, 1e-6, h, y)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(h, want[0]) and torch.equal(y, want[1])

"""add_rmsnorm_dual_out where the sum of squares lies outside fp32: large and tiny streams, infinities,
NaN, and eps at the ends of its range. The formula holds in 64 bits, and so does the kernel's y."""
import numpy as np
import pytest
import torch

from helpers import bf16_ulp
from test_add_rmsnorm_gpu import inputs, mxq  # noqa: F401

pytestmark = pytest.mark.gpu


def run(mxq, x, r, gamma, eps):  # noqa: F811
    T, H = x.shape
    h, y = torch.empty_like(r), torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    yq, rm, tl = torch.empty((T, H), dtype=torch.uint8, device="cuda"), mxq.empty_sf(0, T, H), mxq.empty_sf(2, T, H)
    mxq.add_rmsnorm_dual_out(x, r, gamma, eps, h, y, yq, sf_rowmajor=rm, sf_128x4=tl)
    assert torch.equal(h.nan_to_num(7.0), (x.float() + r.float()).to(r.dtype).nan_to_num(7.0))
    hd, g = h.double().cpu().numpy(), gamma.double().cpu().numpy()
    with np.errstate(all="ignore"):
        ref = hd / np.sqrt((hd * hd).mean(1, keepdims=True) + np.float64(np.float32(eps))) * g
    got = y.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    fin = np.isfinite(ref)
    # the exact value rounded to fp32 and then to bf16 (half a step of each), in bf16's range
    assert (np.abs(got[fin] - ref[fin]) / bf16_ulp(ref[fin])).max(initial=0.0) <= 0.5 + 2.0 ** -16
    q2, rm2, tl2 = torch.empty_like(yq), torch.empty_like(rm), torch.empty_like(tl)
    mxq.mxfp8_quantize(y, q2, rm2, None, tl2)
    assert torch.equal(q2, yq) and torch.equal(rm2, rm) and torch.equal(tl2, tl)
    return got


# every block size of the kernel
SHAPES = [(5, 96), (40, 5120), (600, 512), (520, 5120), (520, 8096), (520, 10240), (520, 16384)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", SHAPES)
def test_large_streams(mxq, T, H, dtype):  # noqa: F811
    x, r, gamma = inputs(T, H, dtype, seed=1)
    scale = torch.ones((T, 1), device="cuda")
    for i, s in enumerate((1e18, 3e18, 1e19, 1e20, 1e30, 1e35, 3e36)):
        scale[i::11] = s
    r = (r.float() * scale).clamp(-3e38, 3e38).to(dtype)
    r[3, 17] = 3e38 if dtype == torch.float32 else torch.finfo(torch.bfloat16).max
    assert np.isfinite(run(mxq, x, r, gamma, 1e-6)).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T,H", SHAPES)
def test_infinities_and_nan(mxq, T, H, dtype):  # noqa: F811
    """One infinity makes its own y NaN and the rest of the row 0; a NaN makes the row NaN."""
    x, r, gamma = inputs(T, H, dtype, seed=2)
    r[0, 5] = float("inf")
    x[2, H - 1] = float("-inf")
    r[4, 0] = float("nan")
    y = run(mxq, x, r, gamma, 1e-6)
    assert np.isnan(y[0]).sum() == 1 and np.isnan(y[2]).sum() == 1 and np.isnan(y[4]).all()
    assert np.isfinite(y[1]).all() and np.isfinite(y[3]).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("eps", [0.0, 1e-38, 1e-25, 1e-6, 1e10, 1e35, 3e38])
def test_tiny_streams_and_eps(mxq, eps, dtype):  # noqa: F811
    T, H = 60, 1024
    x, r, gamma = inputs(T, H, dtype, seed=3)
    scale = torch.ones((T, 1), device="cuda")
    for i, s in enumerate((1e-10, 1e-13, 1e-16, 1e-20, 1e-30)):
        scale[i::7] = s
    x, r = (x.float() * scale).to(torch.bfloat16), (r.float() * scale).to(dtype)
    x[13], r[13] = 0, 0
    y = run(mxq, x, r, gamma, eps)
    assert np.isnan(y[13]).all() if eps == 0.0 else (y[13] == 0).all()

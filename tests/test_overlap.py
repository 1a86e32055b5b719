"""add_rmsnorm_dual_out's check of overlapping arguments: exact for column ranges of one buffer."""
import os
import subprocess

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_against_marked_bytes(tmp_path):
    exe = str(tmp_path / "overlap_check")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-I", os.path.join(ROOT, "mxfp8_activation_quant_gb300", "csrc"),
                    os.path.join(ROOT, "tests", "overlap_check.cpp"), "-o", exe], check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
    apart, _ = map(int, r.stdout.split())
    assert apart > 1000  # cases whose spans meet and whose bytes do not


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_columns_of_one_buffer(dtype):
    """The layer's output and the stream side by side in one buffer, the stream updated in place; and the new
    stream beside the old one."""
    from mxfp8_activation_quant_gb300 import build

    build.build()
    import mxfp8_activation_quant_gb300 as mxq

    T, H = 9, 256
    g = torch.Generator(device="cuda").manual_seed(1)
    gamma = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    buf = torch.randn((T, 3 * H), generator=g, device="cuda").to(dtype)
    x0, r0 = torch.randn((T, H), generator=g, device="cuda").to(torch.bfloat16), buf[:, H:2 * H].clone()
    want, y0 = torch.empty_like(r0), torch.empty_like(x0)
    mxq.add_rmsnorm_dual_out(x0, r0, gamma, 1e-6, want, y0)
    y = torch.empty_like(x0)
    mxq.add_rmsnorm_dual_out(x0, buf[:, H:2 * H], gamma, 1e-6, buf[:, 2 * H:], y)
    assert torch.equal(buf[:, 2 * H:], want) and torch.equal(buf[:, H:2 * H], r0) and torch.equal(y, y0)
    # x as bf16 columns of the same rows
    x = buf.view(torch.bfloat16)[:, :H]
    x.copy_(x0)
    mxq.add_rmsnorm_dual_out(x, buf[:, H:2 * H], gamma, 1e-6, buf[:, H:2 * H], y)
    assert torch.equal(buf[:, H:2 * H], want) and torch.equal(x, x0) and torch.equal(y, y0)
    for out in (buf[:, 2 * H - 8:3 * H - 8], buf[:, 8:H + 8]):  # these do overlap
        with pytest.raises(mxq.MxqError):
            mxq.add_rmsnorm_dual_out(x, buf[:, H:2 * H], gamma, 1e-6, out, y)

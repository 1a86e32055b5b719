"""paged_attention_mxfp8 over values whose scales lie far below others of the same cache head, down to UE8M0's byte 0."""
import pytest
import torch

from kv_reference import attention
from test_paged_attention_gpu import Case, mxq  # noqa: F401  (the module's fixture)

pytestmark = pytest.mark.gpu

ZERO = 448 * 2.0 ** -127  # the largest magnitude of a group of scale byte 0


def values_at(c, scales):
    """The case with one scale byte for each group of features, of every token."""
    for j in range(len(scales)):
        c.vsf[..., j][c.vsf[..., j] != 0xFF] = scales[j]


@pytest.mark.parametrize("scales", [(20, 120, 60, 100), (140, 40, 141, 139), (7, 3, 1, 0), (0, 0, 0, 0), (14, 0, 14, 13)])
@pytest.mark.parametrize("lens", [[200, 90], [5000, 1]])
def test_features_of_far_apart_scales(mxq, scales, lens):  # noqa: F811
    """Up to 2^100 apart each feature has its precision; byte 0 too, where no scale passes 2^-112."""
    c = Case(mxq, lens, 1, 16, 128, False, seed=63)
    values_at(c, scales)
    c.check(c.call(), p_bits=2.0 ** -11 if max(scales) - min(scales) <= 14 else 2.0 ** -8)


@pytest.mark.parametrize("scales", [(0, 118, 0, 117), (0, 16, 0, 16), (118, 0, 60, 118)])
@pytest.mark.parametrize("lens", [[200, 90], [5000, 1]])
def test_byte_0_beside_larger_scales(mxq, scales, lens):  # noqa: F811
    """Its values may count as zeros, and change nothing else."""
    c = Case(mxq, lens, 1, 16, 128, False, seed=64)
    values_at(c, scales)
    out = c.call()["out"]
    o, _, tol, _ = attention(c.q, c.kq, c.ksf, c.vq, c.vsf, c.table, c.lens, c.scale, 2.0 ** -8)
    bound = tol + 2.0 ** -8 * (o.abs() + tol) + 2.0 ** -133
    zero = torch.tensor([s == 0 for s in scales], device="cuda").repeat_interleave(32)
    bound = torch.where(zero, bound + ZERO, bound)
    assert bool(((out.double() - o).abs() <= bound).all())

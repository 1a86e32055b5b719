"""paged_attention_mxfp8 with values next to the largest bf16: no sum on the way to the output may leave fp32."""
import pytest
import torch

from test_paged_attention_gpu import Case, mxq  # noqa: F401  (the module's fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,kv", [([5000], 1), ([20000, 300], 2), ([3000, 2900, 1] * 40, 1), ([1, 64, 200], 1)])
@pytest.mark.parametrize("G,D", [(1, 128), (8, 256), (64, 512)])
def test_values_next_to_the_largest(mxq, lens, kv, G, D):  # noqa: F811
    """Every score 0 and every value 448 * 2^118: so is the output, one CTA's or many parts' (the weights' sum is off by their
    roundings, which the bf16 value's neighbours are further away than)."""
    c = Case(mxq, lens, kv, G, D, False, seed=65, scale=0.0)
    c.vq[c.vsf[..., :1].expand(*c.vsf.shape[:3], D) != 0xFF] = 0x7E
    c.vsf[c.vsf != 0xFF] = 118 + 127
    out = c.call()["out"]
    assert bool((out.double() == 448 * 2.0 ** 118).all())


@pytest.mark.parametrize("lens", [[5000], [3000, 2900] * 50])
def test_large_values_of_both_signs(mxq, lens):  # noqa: F811
    """In 64 bits: values up to 2^126 whose weighted sum is far smaller."""
    c = Case(mxq, lens, 1, 16, 128, False, seed=66)
    c.vsf[c.vsf != 0xFF] = 117 + 127
    pick = [0, len(lens) // 2, len(lens) - 1]
    out = c.call()
    c.q, c.table, c.lens = c.q[pick], c.table[pick], [lens[i] for i in pick]
    c.check(dict(out=out["out"][pick], lse=out["lse"][pick]))

"""paged_attention_mxfp8 whose items are held by several CTAs each, on both sides of where the join changes its form."""
import pytest

from test_paged_attention_gpu import Case, mxq  # noqa: F401  (the module's fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("items", [1, 11, 12, 13, 16, 40, 100])
@pytest.mark.parametrize("G,D,latent", [(8, 128, False), (16, 256, True), (50, 512, True), (64, 384, True)])
def test_parts_of_many_items(mxq, items, G, D, latent):  # noqa: F811
    c = Case(mxq, [max(200, 24000 // items) + 37 * i % 150 for i in range(items)], 1, G, D, latent, seed=67)
    out = c.call(sf=("sf_rowmajor", "sf_packed", "sf_128x4"))
    c.check(out)
    q, sf = mxq.quantize(out["out"].view(items, -1), layouts=(0, 1, 2))
    assert all((a == b).all() for a, b in ((q, out["out_q"]), (sf[0], out["sf_rowmajor"]), (sf[1], out["sf_packed"]), (sf[2], out["sf_128x4"])))

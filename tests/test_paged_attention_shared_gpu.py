"""paged_attention_mxfp8 with a value cache that shares tensors with the key cache: the whole cache, or its scales alone."""
import pytest

from test_paged_attention_gpu import Case, mxq  # noqa: F401  (the module's fixture)

pytestmark = pytest.mark.gpu

LENS = [700, 90, 0, 5000, 129]


class OwnValues(Case):
    """A latent case whose cache is named twice: as the keys and as the values."""

    def caches(self):
        k, _ = super().caches()
        return k, k


@pytest.mark.parametrize("D", [128, 256, 384, 512])
@pytest.mark.parametrize("G", [8, 16, 32, 64])
def test_one_cache_for_both(mxq, G, D):  # noqa: F811
    c = OwnValues(mxq, LENS, 2, G, D, True, page=48, seed=60)
    c.check(c.call())


@pytest.mark.parametrize("D", [128, 256, 384, 512])
@pytest.mark.parametrize("G", [8, 16, 32, 64])
def test_scales_for_both(mxq, G, D):  # noqa: F811
    c = Case(mxq, LENS, 2, G, D, False, page=64, seed=61)
    c.vsf = c.ksf
    c.check(c.call())

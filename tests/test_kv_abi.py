"""include/mxq_kv.h: every declared symbol is exported and bad arguments are refused on the host
(these calls return before any CUDA work, so no GPU is needed)."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x7F0000000000  # never dereferenced: every call below fails validation first
PAGES, PAGE, HEADS, D = 10, 64, 2, 128


@pytest.fixture(scope="module")
def lib():
    from mxfp8_activation_quant_gb300 import build, kv

    build.build()
    return kv._fns()


def cache(**kw):
    from mxfp8_activation_quant_gb300.kv import _CACHE

    a = dict(data=FAKE, sf=FAKE, pages=PAGES, page_size=PAGE, heads=HEADS, dim=D, page_stride=PAGE * HEADS * D,
             token_stride=HEADS * D, head_stride=D, sf_page_stride=PAGE * HEADS * D // 32,
             sf_token_stride=HEADS * D // 32, sf_head_stride=D // 32)
    a.update(kw)
    return _CACHE.pack(*(v or 0 for v in a.values()))


BAD_CACHES = [
    (dict(data=None), 1), (dict(sf=None), 1), (dict(pages=0), 1), (dict(page_size=0), 1), (dict(heads=0), 1), (dict(dim=0), 1),
    (dict(pages=-1), 1), (dict(dim=100), 2), (dict(dim=1056), 2), (dict(heads=1025), 2), (dict(page_size=65552), 2),
    (dict(pages=2 ** 31), 2), (dict(pages=2 ** 25), 2),              # 2^31 slots
    (dict(page_stride=2 ** 40), 2), (dict(token_stride=-256), 2), (dict(sf_page_stride=2 ** 40), 2),
    (dict(data=FAKE + 8), 3), (dict(sf=FAKE + 2), 3), (dict(token_stride=HEADS * D + 8), 3), (dict(head_stride=D + 8), 3),
    (dict(page_stride=PAGE * HEADS * D + 8), 3), (dict(sf_head_stride=6), 3), (dict(sf_token_stride=10), 3),
    (dict(head_stride=64), 1), (dict(token_stride=D), 1), (dict(page_stride=D), 1),   # rows that overlap
    (dict(token_stride=0), 1), (dict(sf_token_stride=4), 1), (dict(page_stride=PAGE * HEADS * D - 16), 1),
]


def ref(c):
    return c  # (the struct's bytes, or None)


def write(lib, kc=None, vc=None, k=FAKE, ldk=HEADS * D, ldkh=D, v=None, ldv=HEADS * D, ldvh=D, slots=FAKE, T=4):
    return lib.kv_write_mxfp8(k, ldk, ldkh, ref(kc), v, ldv, ldvh, ref(vc), slots, T, None)


def read(lib, kc=None, vc=None, table=FAKE, ldt=8, width=8, cu=FAKE, starts=None, B=4, rows=100, ko=FAKE, vo=None):
    return lib.kv_read_bf16(ref(kc), ref(vc), table, ldt, width, cu, starts, B, rows, ko, vo, None)


def attend(lib, kc=None, vc=None, q=FAKE, ldq=16 * D, ldqh=D, table=FAKE, ldt=8, width=8, lens=FAKE, B=4, H=16, scale=0.1,
           o=FAKE, oq=None, pk=None, rm=None, tl=None, lse=None, ws=FAKE, wsn=None, st=None):
    if wsn is None:
        wsn = 1 << 60  # (never looked into)
    return lib.paged_attention_mxfp8(q, ldq, ldqh, ref(kc), ref(vc), table, ldt, width, lens, B, H, scale, o, oq, pk, rm,
                                     tl, lse, ws, wsn, st, None)


def test_every_declared_symbol_is_exported(lib):
    from mxfp8_activation_quant_gb300 import kv

    text = open(os.path.join(ROOT, "include", "mxq_kv.h")).read()
    names = re.findall(r"MXQ_API\s+[\w\s\*]+?\b(\w+)\s*\(", text)
    assert set(names) == set(kv.SIGNATURES) and len(names) == 4
    for n in names:
        assert hasattr(lib, n), n


@pytest.mark.parametrize("change,status", BAD_CACHES)
def test_cache_refusals(lib, change, status):
    bad, good = cache(**change), cache()
    assert write(lib, bad) == status and read(lib, bad) == status and attend(lib, bad) == status
    assert write(lib, good, bad, v=FAKE) == status and read(lib, good, bad, vo=FAKE) == status
    assert attend(lib, good, bad) == status


def test_strides_of_single_dimensions_are_not_looked_at(lib):
    """A good cache with senseless strides where a size is 1 gets past the cache's checks (T = 0 ends the call)."""
    c = cache(heads=1, head_stride=7, sf_head_stride=-3)
    assert write(lib, c, k=None) == 1 and write(lib, c, ldk=D - 8) == 2  # (refused for the rows, not the cache)
    c = cache(pages=1, page_stride=3, sf_page_stride=2 ** 50)
    assert write(lib, c, ldk=D - 8) == 2


def test_write_refusals(lib):
    c = cache()
    assert write(lib, None) == 1 and write(lib, c, k=None) == 1 and write(lib, c, slots=None) == 1
    assert write(lib, c, T=0) == 1 and write(lib, c, T=-4) == 1 and write(lib, c, T=2 ** 31) == 2
    assert write(lib, c, c, v=None) == 1 and write(lib, c, None, v=FAKE) == 1
    assert write(lib, c, ldk=D - 8) == 2 and write(lib, c, ldkh=D - 8) == 2 and write(lib, c, ldk=2 ** 40) == 2
    assert write(lib, c, ldk=2 * D + 4) == 3 and write(lib, c, ldkh=D + 4) == 3 and write(lib, c, k=FAKE + 2) == 3
    assert write(lib, c, slots=FAKE + 2) == 3 and write(lib, c, c, v=FAKE + 8) == 3
    assert write(lib, c, cache(pages=9), v=FAKE) == 2 and write(lib, c, cache(page_size=32), v=FAKE) == 2


def test_read_refusals(lib):
    c = cache()
    assert read(lib, None) == 1 and read(lib, c, table=None) == 1 and read(lib, c, cu=None) == 1 and read(lib, c, ko=None) == 1
    assert read(lib, c, B=0) == 1 and read(lib, c, rows=0) == 1 and read(lib, c, width=0) == 1
    assert read(lib, c, c, vo=None) == 1 and read(lib, c, None, vo=FAKE) == 1
    assert read(lib, c, ldt=7) == 2 and read(lib, c, rows=2 ** 31) == 2 and read(lib, c, cache(pages=11), vo=FAKE) == 2
    assert read(lib, c, table=FAKE + 2) == 3 and read(lib, c, cu=FAKE + 1) == 3 and read(lib, c, starts=FAKE + 2) == 3
    assert read(lib, c, ko=FAKE + 8) == 3


def test_attention_refusals(lib):
    c = cache()
    for name in ("q", "table", "lens", "ws"):
        assert attend(lib, c, **{name: None}) == 1, name
    assert attend(lib, None) == 1 and attend(lib, c, o=None) == 1 and attend(lib, c, o=None, rm=FAKE) == 1
    assert attend(lib, c, oq=FAKE) == 1 and attend(lib, c, rm=FAKE) == 1      # o_q without scales, scales without o_q
    assert attend(lib, c, B=0) == 1 and attend(lib, c, H=0) == 1 and attend(lib, c, width=0) == 1
    assert attend(lib, c, scale=float("nan")) == 1 and attend(lib, c, scale=float("inf")) == 1
    assert attend(lib, c, wsn=0) == 1
    assert attend(lib, c, H=15) == 2 and attend(lib, c, H=4098, ldq=4098 * D) == 2 and attend(lib, c, B=32769) == 2
    assert attend(lib, c, ldq=D - 8) == 2 and attend(lib, c, ldqh=D - 8) == 2 and attend(lib, c, ldt=7) == 2
    for dim in (32, 64, 96, 192, 640):
        k = cache(dim=dim, head_stride=1024, token_stride=2048, page_stride=2048 * PAGE, sf_head_stride=32, sf_token_stride=64,
                  sf_page_stride=64 * PAGE)
        assert attend(lib, k, ldq=16 * dim, ldqh=dim) == 2, dim
    assert attend(lib, cache(page_size=40)) == 2
    for change in (dict(pages=9), dict(page_size=48), dict(heads=1)):
        assert attend(lib, c, cache(**change)) == 2, change
    assert attend(lib, c, ldq=16 * D + 4) == 3 and attend(lib, c, q=FAKE + 2) == 3 and attend(lib, c, o=FAKE + 2) == 3
    assert attend(lib, c, oq=FAKE + 8, rm=FAKE) == 3 and attend(lib, c, oq=FAKE, tl=FAKE + 8) == 3
    assert attend(lib, c, lse=FAKE + 2) == 3 and attend(lib, c, lens=FAKE + 2) == 3 and attend(lib, c, table=FAKE + 2) == 3
    assert attend(lib, c, ws=FAKE + 8) == 3 and attend(lib, c, st=FAKE + 8) == 3


def test_workspace_of_invalid_shapes_is_zero(lib):
    w = lib.mxq_paged_attention_workspace_bytes
    assert w(0, 16, 2, 128) == 0 and w(4, 0, 2, 128) == 0 and w(4, 16, 0, 128) == 0 and w(4, 16, 3, 128) == 0
    assert w(4, 16, 2, 64) == 0 and w(4, 4098, 2, 128) == 0 and w(32769, 16, 2, 128) == 0
    assert w(4, 16, 2, 128) > 0 and w(65536, 1, 1, 128) % 16 == 0


def test_host_tensors_and_wrong_types_are_refused(lib):
    """The binding passes device pointers only: a host tensor is an error, not a CPU path."""
    import torch

    from mxfp8_activation_quant_gb300 import kv

    c = kv.MXFP8Cache.empty(4, 16, 2, 128, device="cpu")
    k, slots = torch.zeros(3, 2, 128, dtype=torch.bfloat16), torch.zeros(3, dtype=torch.int32)
    table, lens = torch.zeros(3, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    q = torch.zeros(3, 16, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensors"):
        kv.kv_write_mxfp8(k, slots, c)
    with pytest.raises(ValueError, match="device tensors"):
        kv.kv_read_bf16(c, table, torch.zeros(4, dtype=torch.int32), k)
    with pytest.raises(ValueError, match="device tensors"):
        kv.paged_attention_mxfp8(q, c, table, lens, 0.1, out=torch.empty_like(q))
    with pytest.raises(AssertionError):
        kv.kv_write_mxfp8(k, slots.long(), c)
    with pytest.raises(AssertionError):
        kv.kv_write_mxfp8(k.float(), slots, c)
    with pytest.raises(AssertionError):
        kv.kv_write_mxfp8(k, slots, c, v=k)
    with pytest.raises(AssertionError):
        kv.MXFP8Cache(c.data, c.sf[..., :2]).c()
    with pytest.raises(AssertionError):
        kv.paged_attention_mxfp8(q, c, table, lens.long(), 0.1, out=torch.empty_like(q))
    for name, n in (("sf_rowmajor", 3 * 64), ("sf_packed", 4 * 64), ("sf_128x4", 128 * 64)):
        with pytest.raises(AssertionError):
            kv.paged_attention_mxfp8(q, c, table, lens, 0.1, out_q=torch.zeros(3, 2048, dtype=torch.uint8),
                                     **{name: torch.zeros(n - 4, dtype=torch.uint8)})


def test_limits_of_lengths_strides_and_scale(lib):
    c = cache()
    assert attend(lib, c, B=1, width=2 ** 24 + 1, ldt=2 ** 25) == 2          # 2^30 + 64 places
    wide = cache(pages=2 ** 20, page_size=16)
    # pieces of 64 tokens: 512 sequences x 2 cache heads x 2^20 = 2^30; one sequence less passes (wsn = 0 then ends the call)
    assert attend(lib, wide, B=512, width=2 ** 22, ldt=2 ** 22) == 2
    assert attend(lib, wide, B=511, width=2 ** 22, ldt=2 ** 22, wsn=0) == 1
    # and blocks of 64 query heads count: 65 a cache head are two
    assert attend(lib, wide, B=256, H=130, ldq=130 * D, width=2 ** 22, ldt=2 ** 22) == 2
    for s in (2e38, -2e38):
        assert attend(lib, c, scale=s) == 1
    assert attend(lib, c, scale=-1e38, wsn=0) == 1 and attend(lib, c, scale=1e38, lse=FAKE + 2) == 3
    assert attend(lib, cache(sf_page_stride=2 ** 31)) == 2 and write(lib, cache(sf_page_stride=2 ** 31)) == 2

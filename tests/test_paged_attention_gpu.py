"""paged_attention_mxfp8 against the definition in 64 bits (kv_reference.attention, which derives the tolerances)."""
import math

import pytest
import torch

from kv_reference import attention, empty_cache, fill, pages_for, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mxq():
    from mxfp8_activation_quant_gb300 import build

    build.build()
    import mxfp8_activation_quant_gb300 as m

    assert torch.cuda.is_available(), "GPU tests need CUDA"
    m.load()
    return m


class Case:
    def __init__(self, mxq, lens, kv, G, D, latent, page=64, order="nhd", seed=0, width=None, scale=None, mean=116, spread=2, q_stride=None):
        self.m, self.lens, self.kv, self.G, self.D = mxq, lens, kv, G, D
        g = self.g = torch.Generator(device="cuda").manual_seed(seed + 1000 * D + 7 * G + len(lens))
        B, H = len(lens), kv * G
        self.table, pages = pages_for(g, lens, page, width=width)
        self.kq, self.ksf = empty_cache(pages, page, kv, D, order)
        fill(g, self.kq, self.ksf, self.table, lens, mean, spread)
        self.vq = self.vsf = None
        if not latent:
            self.vq, self.vsf = empty_cache(pages, page, kv, D, order, pad=2)
            fill(g, self.vq, self.vsf, self.table, lens, mean, spread)
        q = torch.randn((B, H, D), generator=g, device="cuda").to(torch.bfloat16)
        if q_stride:  # heads and sequences further apart, NaN between them
            wide = torch.full((B, H + 1, D + q_stride), math.nan, dtype=torch.bfloat16, device="cuda")
            self.q = wide[:, :H, :D]
            self.q.copy_(q)
        else:
            self.q = q
        # codes are spread evenly over their exponents: rms about 2^6.1; scores of a few units
        self.scale = 2.0 / (math.sqrt(D) * 70 * 2.0 ** (mean - 127)) if scale is None else scale
        self.seq = torch.tensor(lens, dtype=torch.int32, device="cuda")

    def caches(self):
        k = self.m.MXFP8Cache(self.kq, self.ksf)
        return k, None if self.vq is None else self.m.MXFP8Cache(self.vq, self.vsf)

    def call(self, sf=None, bf16=True, lse=True, stream=None, workspace=None):
        m, (B, H, D) = self.m, self.q.shape
        k, v = self.caches()
        out = dict(out=torch.full((B, H, D), math.nan, dtype=torch.bfloat16, device="cuda")) if bf16 else {}
        if lse:
            out["lse"] = torch.full((B, H), math.nan, device="cuda")
        if sf is not None:
            out["out_q"] = torch.full((B, H * D), 0x7F, dtype=torch.uint8, device="cuda")
            for name, layout in (("sf_rowmajor", 0), ("sf_packed", 1), ("sf_128x4", 2)):
                if name in sf:
                    out[name] = m.empty_sf(layout, B, H * D).fill_(0xEE)
        status = m.new_status()
        m.paged_attention_mxfp8(self.q, k, self.table, self.seq, self.scale, v_cache=v, status=status, stream=stream,
                                workspace=workspace, **out)
        m.check_status(status, stream)
        return out

    def check(self, out, p_bits=2.0 ** -11):
        o, lse, tol, ltol = attention(self.q, self.kq, self.ksf, self.vq, self.vsf, self.table, self.lens, self.scale, p_bits)
        err = (out["out"].double() - o).abs()
        # one rounding to bf16: half a step is 2^-8 of the value that is rounded, which is within tol of o
        bound = tol + 2.0 ** -8 * (o.abs() + tol) + 2.0 ** -133
        assert bool((err <= bound).all()), f"off by {float((err / bound.clamp_min(1e-300)).max())} of the tolerance"
        if "lse" in out:
            assert torch.equal(out["lse"].isinf(), lse.isinf())
            le = torch.where(lse.isinf(), 0.0, (out["lse"].double() - lse).abs())
            assert bool((le <= ltol).all()), f"lse off by {float((le / ltol.clamp_min(1e-300)).max())} of the tolerance"


EDGES = [0, 1, 15, 16, 17, 63, 64, 65, 127, 128, 129, 191, 300]


@pytest.mark.parametrize("kv,G,D,latent,page,order", [
    (1, 64, 512, True, 64, "nhd"), (1, 16, 128, True, 16, "nhd"), (1, 64, 256, False, 48, "hnd"), (2, 8, 128, False, 16, "hnd"),
    (1, 128, 384, True, 80, "nhd"), (3, 3, 256, False, 32, "nhd"), (5, 1, 128, False, 128, "hnd"), (1, 33, 512, False, 256, "nhd"),
    (2, 65, 128, False, 112, "nhd"), (1, 24, 384, True, 1040, "nhd"),
])
def test_lengths(mxq, kv, G, D, latent, page, order):
    c = Case(mxq, EDGES, kv, G, D, latent, page, order)
    out = c.call()
    c.check(out)
    assert not out["out"][0].any()  # a sequence without a token: zeros


@pytest.mark.parametrize("lens,kv,G,D,latent", [
    ([5000], 1, 64, 512, True), ([20011], 2, 8, 128, False), ([3, 7000, 0, 2500], 1, 40, 256, False), ([1], 1, 1, 128, True),
    ([700] * 40 + [1] * 200 + [0] * 33, 2, 4, 128, False), ([400, 10] * 100, 1, 64, 512, True),
])
def test_long_and_many(mxq, lens, kv, G, D, latent):
    c = Case(mxq, lens, kv, G, D, latent, page=64, seed=5)
    c.check(c.call())


@pytest.mark.parametrize("B", [1, 3, 4, 5, 130])
@pytest.mark.parametrize("kv,G,D,latent", [(1, 64, 512, True), (3, 4, 128, False)])
def test_mxfp8_output(mxq, B, kv, G, D, latent):
    """o_q and its scales are mxfp8_quantize(o), in every layout and with their padding; o alone or o_q alone are the same."""
    c = Case(mxq, [(37 * i) % 150 for i in range(B)], kv, G, D, latent, seed=B)
    out = c.call(sf=("sf_rowmajor", "sf_packed", "sf_128x4"))
    c.check(out)
    q, sf = mxq.quantize(out["out"].view(B, -1), layouts=(0, 1, 2))
    assert torch.equal(q, out["out_q"])
    assert torch.equal(sf[0], out["sf_rowmajor"]) and torch.equal(sf[1], out["sf_packed"]) and torch.equal(sf[2], out["sf_128x4"])
    only = c.call(sf=("sf_128x4",), bf16=False, lse=False)
    assert torch.equal(only["out_q"], q) and torch.equal(only["sf_128x4"], sf[2])
    assert torch.equal(c.call(lse=False)["out"], out["out"])


def test_pages_outside_the_cache(mxq):
    """Tokens on a page outside [0, pages) take no part; a sequence with no other gives zeros."""
    c = Case(mxq, [300, 64, 200, 500], 2, 8, 128, False, page=16, seed=1)
    c.table[0, 3] = -1
    c.table[0, 7] = c.kq.shape[0]
    c.table[1, :] = 2 ** 31 - 1
    c.table[2, :12] = -2 ** 31
    c.table[3, 31] = c.kq.shape[0] + 5
    out = c.call()
    c.check(out)
    assert not out["out"][1].any() and bool((out["lse"][1] == -math.inf).all())


def test_lengths_past_the_table_and_below_zero(mxq):
    c = Case(mxq, [128, 100, 64], 1, 16, 256, True, page=64, seed=2)
    c.lens = [1000, -5, 2 ** 31 - 1]
    c.seq = torch.tensor(c.lens, dtype=torch.int32, device="cuda")
    # the table's pages past the filled ones hold NaN, so the table is cut to what is filled
    c.table = c.table[:, :1].contiguous()
    out = c.call()
    c.check(out)
    assert not out["out"][1].any()


def test_strided_queries_and_tables(mxq):
    c = Case(mxq, [90, 200, 31], 2, 5, 128, False, q_stride=64, seed=3)
    wide = torch.full((3, c.table.shape[1] + 9), -1, dtype=torch.int32, device="cuda")
    wide[:, :c.table.shape[1]] = c.table
    c.table = wide[:, :c.table.shape[1]]
    c.check(c.call())


def test_keys_and_values_in_one_buffer(mxq):
    """A page holds keys then values (strides with other data between), pages of several sequences shared."""
    g = torch.Generator(device="cuda").manual_seed(4)
    q = torch.full((9, 2, 32, 3, 128), 0x7F, dtype=torch.uint8, device="cuda")
    sf = torch.full((9, 2, 32, 3, 4), 0xFF, dtype=torch.uint8, device="cuda")
    c = Case(mxq, [70, 70, 40], 3, 6, 128, False, page=32)
    c.kq, c.vq, c.ksf, c.vsf = q[:, 0], q[:, 1], sf[:, 0], sf[:, 1]
    c.table = torch.tensor([[5, 1, 7], [5, 1, 8], [5, 1, 0]], dtype=torch.int32, device="cuda")  # a common prefix
    for x, s in ((c.kq, c.ksf), (c.vq, c.vsf)):
        fill(g, x, s, c.table, [70, 70, 40], 116, 2)
    c.check(c.call())


@pytest.mark.parametrize("kv,G,D,latent", [(1, 64, 512, True), (2, 8, 128, False)])
def test_rising_and_falling_scores(mxq, kv, G, D, latent):
    """The largest score keeps rising from tile to tile, or lies at the start: sums are carried through it."""
    for order in (1, -1):
        c = Case(mxq, [900, 2000], kv, G, D, latent, seed=6)
        c.q.copy_(c.q.abs())
        for b, n in enumerate(c.lens):
            for j in range(-(-n // 64)):
                p = int(c.table[b, j])
                m = min(64, n - j * 64)
                k = c.kq[p, :m] & 0x7F  # positive keys, growing along the sequence
                c.kq[p, :m] = k
                tokens = torch.arange(j * 64, j * 64 + m, device="cuda")
                step = (tokens if order > 0 else n - tokens) // 300
                c.ksf[p, :m] = (112 + step).to(torch.uint8).view(m, 1, 1)
        c.scale = 1.0 / (D * 60 * 2.0 ** (112 - 127)) * 8
        c.check(c.call())


@pytest.mark.parametrize("latent", [True, False])
def test_one_token_takes_all(mxq, latent):
    """A score far above the others at the first, a middle and the last token."""
    for at in (0, 70, 399):
        c = Case(mxq, [400], 1, 16, 256, latent, seed=8 + at)
        p = int(c.table[0, at // 64])
        c.kq[p, at % 64] = 0x38 + torch.zeros(256, dtype=torch.uint8, device="cuda")  # 1.0
        c.ksf[p, at % 64] = 127
        c.q.copy_(c.q.abs())
        c.scale = 3.0
        c.check(c.call())


@pytest.mark.parametrize("kv,G,D", [(1, 32, 512), (2, 8, 128)])
def test_values_of_far_apart_scales(mxq, kv, G, D):
    """Scales of the values that span more than fp16 holds, within a tile and between tiles; all-zero tokens."""
    c = Case(mxq, [700, 90], kv, G, D, False, seed=9)
    for b, n in enumerate(c.lens):
        for j in range(-(-n // 64)):
            p, m = int(c.table[b, j]), min(64, n - j * 64)
            c.vsf[p, :m] = torch.randint(60, 200, (m, kv, D // 32), generator=c.g, device="cuda").to(torch.uint8)
            c.vq[p, 0], c.vsf[p, 0] = 0, 0
    c.check(c.call(), p_bits=2.0 ** -8)
    # one far larger token in a later tile only
    c = Case(mxq, [700], kv, G, D, False, seed=10)
    c.vsf[int(c.table[0, 6]), 10] = 160
    c.check(c.call(), p_bits=2.0 ** -8)
    # and values next to nothing after large ones
    c = Case(mxq, [700], kv, G, D, False, seed=11)
    for j in range(3, 11):
        c.vsf[int(c.table[0, j]), :min(64, 700 - j * 64)] = 80
    c.check(c.call(), p_bits=2.0 ** -8)


def test_extreme_scales(mxq):
    """The ends of UE8M0's range: keys and values next to the smallest and the largest."""
    for kmean, vmean, qe in ((20, 20, 100), (225, 225, -90), (1, 240, 110)):
        c = Case(mxq, [150, 33], 1, 16, 128, False, mean=kmean, spread=0, seed=12)
        c.vsf[c.vsf != 0xFF] = vmean
        c.q.copy_((c.q.float() * 2.0 ** qe).to(torch.bfloat16))
        # scores of a few units, in steps that fp32 holds
        c.scale = 2.0 / (math.sqrt(128) * 70) * 2.0 ** (127 - kmean - qe)
        c.check(c.call())


@pytest.mark.parametrize("scale", [0.0, -0.02])
def test_zero_and_negative_scale(mxq, scale):
    c = Case(mxq, [200, 1, 77], 1, 20, 128, False, seed=13, scale=scale, mean=120)
    c.check(c.call())


def test_queries_of_mixed_magnitudes(mxq):
    """Groups of q with one large element beside small ones, and all-zero groups and heads."""
    c = Case(mxq, [150, 260], 1, 64, 512, True, seed=14)
    q = c.q.float() * torch.exp2(torch.randint(-12, 3, c.q.shape, generator=c.g, device="cuda").float())
    q[:, 3] = 0
    q[:, :, 64:96] = 0
    c.q.copy_(q.to(torch.bfloat16))
    c.check(c.call())


def test_repeated_calls_are_equal(mxq):
    c = Case(mxq, [5000, 100, 2000], 1, 64, 512, True, seed=15)
    a = c.call(sf=("sf_128x4",))
    for _ in range(3):
        b = c.call(sf=("sf_128x4",))
        assert all(torch.equal(a[k], b[k]) for k in a)


def test_dirty_workspace(mxq):
    c = Case(mxq, [5000, 100, 0], 2, 8, 128, False, seed=16)
    a = c.call()
    n = mxq.paged_attention_workspace_bytes(3, 16, 2, 128)
    ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")
    assert torch.equal(c.call(workspace=ws)["out"], a["out"])


def test_captured_and_replayed(mxq):
    """A graph of the call, replayed with other lengths, queries and pages; beside an eager call on another stream."""
    c = Case(mxq, [3000, 700, 64], 2, 8, 128, False, seed=17)
    k, v = c.caches()
    out, lse = torch.empty_like(c.q), torch.empty((3, 16), device="cuda")
    ws = torch.empty(mxq.paged_attention_workspace_bytes(3, 16, 2, 128), dtype=torch.uint8, device="cuda")

    def step():
        mxq.paged_attention_mxfp8(c.q, k, c.table, c.seq, c.scale, v_cache=v, out=out, lse=lse, workspace=ws)

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    other = Case(mxq, [900, 901], 1, 64, 512, True, seed=18)
    want = other.call()["out"]
    side = torch.cuda.Stream()
    for lens in ([1, 0, 64], [3000, 64, 13], [17, 700, 5]):
        c.lens = lens
        c.seq.copy_(torch.tensor(lens, dtype=torch.int32))
        c.q.copy_(torch.randn(c.q.shape, generator=c.g, device="cuda").to(torch.bfloat16))
        torch.cuda.synchronize()
        graph.replay()
        beside = other.call(stream=side)["out"]
        torch.cuda.synchronize()
        c.check(dict(out=out, lse=lse))
        assert torch.equal(beside, want)


def test_past_32_bits(mxq):
    """Pages more than 2^32 bytes into the cache."""
    pages, page, D = 150000, 64, 512
    c = Case(mxq, [100, 64], 1, 64, D, True, seed=19)
    q = torch.empty((pages, page, 1, D), dtype=torch.uint8, device="cuda")
    sf = torch.empty((pages, page, 1, D // 32), dtype=torch.uint8, device="cuda")
    table = torch.tensor([[pages - 1, 140000], [141111, 0]], dtype=torch.int32, device="cuda")
    for p in (pages - 1, 140000, 141111):
        q[p], sf[p] = 0x7F, 0xFF
    fill(c.g, q, sf, table, [100, 64], 116, 2)
    c.kq, c.ksf, c.table = q, sf, table
    c.check(c.call())


def test_a_status_word_stays_clear_and_scores_are_used(mxq):
    """Not the mean of the values: with equal keys it is that."""
    c = Case(mxq, [130], 1, 8, 128, False, seed=20)
    p = c.table[0].long()
    c.kq[p], c.ksf[p] = 0x30, 120
    out = c.call()["out"]
    v = values(c.vq[p].reshape(-1, 1, 128)[:130], c.vsf[p].reshape(-1, 1, 4)[:130]).mean(0)
    assert bool(((out[0].double() - v).abs() <= 2.0 ** -8 * v.abs() + 2.0 ** -10 * 448 * 2.0 ** -9).all())

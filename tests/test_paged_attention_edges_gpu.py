"""paged_attention_mxfp8 where kinds of calls meet: every padded number of heads with every number of features, NaN among
the tokens, outputs over the queries, streams, graphs and threads that keep their own workspaces."""
import math
import threading

import pytest
import torch

from kv_reference import empty_cache, fill
from test_paged_attention_gpu import Case, mxq  # noqa: F401  (the module's fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("latent", [True, False])
@pytest.mark.parametrize("D", [128, 256, 384, 512])
@pytest.mark.parametrize("G", [5, 13, 27, 50, 100])
def test_every_kernel(mxq, G, D, latent):  # noqa: F811
    """Items of one CTA and of several, bf16 and MXFP8 from one call."""
    c = Case(mxq, [3000, 40, 0, 333, 129], 2, G, D, latent, page=16, seed=30)
    out = c.call(sf=("sf_rowmajor", "sf_packed", "sf_128x4"))
    c.check(out)
    q, sf = mxq.quantize(out["out"].view(5, -1), layouts=(0, 1, 2))
    assert torch.equal(q, out["out_q"])
    assert torch.equal(sf[0], out["sf_rowmajor"]) and torch.equal(sf[1], out["sf_packed"]) and torch.equal(sf[2], out["sf_128x4"])


@pytest.mark.parametrize("G,D,latent", [(64, 512, True), (8, 512, False), (16, 384, False)])
def test_scales_on_words_only(mxq, G, D, latent):  # noqa: F811
    """Rows of scales that start on 4-byte boundaries and no wider ones."""
    c = Case(mxq, [400, 70], 1, G, D, latent, seed=31)
    want = c.call()
    for name in ("ksf", "vsf"):
        sf = getattr(c, name)
        if sf is not None:
            wide = torch.full((*sf.shape[:3], D // 32 + 4), 0xFF, dtype=torch.uint8, device="cuda")
            wide[..., 4:] = sf
            setattr(c, name, wide[..., 4:])
    got = c.call()
    assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"])


@pytest.mark.parametrize("lens", [[200, 90, 130], [5000, 300, 2000]])
def test_nan_among_the_tokens(mxq, lens):  # noqa: F811
    """NaN reaches its own sequence's cache head, or there its own feature, and nothing else."""
    c = Case(mxq, lens, 2, 8, 128, False, seed=32)
    clean = c.call()
    at = lambda t: (int(c.table[1, t // 64]), t % 64)  # noqa: E731
    heads = slice(8, 16)  # of cache head 1

    def planted(cache, value, t, *where):
        p, r = at(t)
        old = cache[(p, r, 1, *where)].clone()
        cache[(p, r, 1, *where)] = value
        out = c.call()
        cache[(p, r, 1, *where)] = old
        return out

    def agree(out, nan, lse_nan):
        assert torch.equal(out["out"].isnan(), nan)
        assert torch.equal(torch.where(nan, 0, out["out"]), torch.where(nan, 0, clean["out"]))
        assert torch.equal(out["lse"].isnan(), lse_nan)
        assert torch.equal(torch.where(lse_nan, 0, out["lse"]), torch.where(lse_nan, 0, clean["lse"]))

    none = torch.zeros_like(clean["out"], dtype=torch.bool)
    own, own_lse = none.clone(), torch.zeros_like(clean["lse"], dtype=torch.bool)
    own[1, heads] = True
    own_lse[1, heads] = True
    feature = none.clone()
    feature[1, heads, 77] = True
    for t in (0, 70, 89):
        agree(planted(c.kq, 0x7F, t, 5), own, own_lse)
        agree(planted(c.ksf, 0xFF, t, 2), own, own_lse)
        agree(planted(c.vq, 0xFF, t, 77), feature, torch.zeros_like(own_lse))
        agree(planted(c.vsf, 0xFF, t, 2), own, torch.zeros_like(own_lse))


def test_scores_next_to_the_lowest(mxq):  # noqa: F811
    """Equal scores of about -2^120: the mean of the values, and lse that score plus ln n (2^-22 of it, next to which ln n is
    nothing)."""
    c = Case(mxq, [150], 1, 8, 128, False, seed=33, scale=1.0)
    c.kq[c.table[0].long()], c.ksf[c.table[0].long()] = 0x38, 127 + 60  # 2^60
    c.q.fill_(-2.0 ** 53)                                              # 128 products of -2^113
    got = c.call()
    c.scale, c.q = 0.0, torch.zeros_like(c.q)
    c.check(dict(out=got["out"]))
    assert bool(((got["lse"].double() + 2.0 ** 120).abs() <= 2.0 ** (120 - 22)).all())


@pytest.mark.parametrize("lens,kv,G,D,latent", [([4000, 100], 1, 64, 512, True), ([30, 0, 64], 2, 8, 128, False)])
def test_output_over_the_queries(mxq, lens, kv, G, D, latent):  # noqa: F811
    c = Case(mxq, lens, kv, G, D, latent, seed=34)
    want = c.call()["out"]
    k, v = c.caches()
    mxq.paged_attention_mxfp8(c.q, k, c.table, c.seq, c.scale, v_cache=v, out=c.q)
    assert torch.equal(c.q, want)


def test_many_sequences(mxq):  # noqa: F811
    """More sequences than threads of a CTA, most with a few tokens."""
    lens = [(7919 * i) % 23 for i in range(3000)]
    lens[1234] = 700
    c = Case(mxq, lens, 2, 2, 128, False, page=16, width=44, seed=35)
    out = c.call(sf=("sf_128x4",))
    pick = list(range(0, 3000, 61)) + [1234]
    o = out["out"]
    c.q, c.table, c.lens = c.q[pick], c.table[pick], [lens[i] for i in pick]
    c.check(dict(out=o[pick], lse=out["lse"][pick]))
    q, sf = mxq.quantize(o.view(3000, -1), layouts=(2,))
    assert torch.equal(q, out["out_q"]) and torch.equal(sf[2], out["sf_128x4"])


def two_cases(mxq):  # noqa: F811
    return (Case(mxq, [3000, 700, 64], 2, 8, 128, False, seed=36), Case(mxq, [2000, 901], 1, 64, 512, True, seed=37))


def test_two_graphs_without_a_workspace_argument(mxq):  # noqa: F811
    """Each graph has a workspace of its own: replayed at once on two streams, beside eager calls on a third."""
    cases = two_cases(mxq)
    want = [c.call()["out"] for c in cases]
    outs, graphs = [torch.empty_like(c.q) for c in cases], []
    for c, out in zip(cases, outs):
        k, v = c.caches()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            mxq.paged_attention_mxfp8(c.q, k, c.table, c.seq, c.scale, v_cache=v, out=out)
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for o in outs:
            o.fill_(math.nan)
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        eager = cases[0].call()["out"]
        torch.cuda.synchronize()
        assert torch.equal(eager, want[0]) and all(torch.equal(o, w) for o, w in zip(outs, want))


def test_captured_on_a_stream_that_is_named(mxq):  # noqa: F811
    """stream= under capture: the workspace is the graph's, whichever stream is the current one."""
    c, other = two_cases(mxq)
    want = c.call()["out"]
    k, v = c.caches()
    out, s = torch.empty_like(c.q), torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        mxq.paged_attention_mxfp8(c.q, k, c.table, c.seq, c.scale, v_cache=v, out=out, stream=s.cuda_stream)
    other.call(stream=s)  # (grows what is kept for the stream)
    for _ in range(3):
        out.fill_(math.nan)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_two_threads_on_one_stream(mxq):  # noqa: F811
    """They share the stream's workspace, so a call's launches are not mixed with another's."""
    cases = two_cases(mxq)
    want = [c.call()["out"] for c in cases]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        c, (k, v) = cases[i], cases[i].caches()
        outs = [torch.empty_like(c.q) for _ in range(60)]
        for out in outs:
            mxq.paged_attention_mxfp8(c.q, k, c.table, c.seq, c.scale, v_cache=v, out=out)
        torch.cuda.synchronize()
        bad.extend(i for out in outs if not torch.equal(out, want[i]))

    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


def test_lengths_change_what_a_workspace_held(mxq):  # noqa: F811
    """Calls of many shapes on one stream, one after another without a wait: what one leaves in the workspace does
    not matter to the next."""
    shapes = [([5000], 1, 64, 512, True), ([1, 0], 2, 3, 128, False), ([800] * 30, 2, 8, 128, False), ([64], 1, 33, 256, True)]
    cases = [Case(mxq, *s, seed=38 + i) for i, s in enumerate(shapes)]
    want = [c.call()["out"] for c in cases]
    got = []
    for i in (0, 1, 2, 3, 2, 1, 0, 3, 1, 0, 2):
        c = cases[i]
        k, v = c.caches()
        out = torch.empty_like(c.q)
        mxq.paged_attention_mxfp8(c.q, k, c.table, c.seq, c.scale, v_cache=v, out=out)
        got.append((i, out))
    assert all(torch.equal(out, want[i]) for i, out in got)


def test_interleaved_page_orders(mxq):  # noqa: F811
    """Keys by tokens, values by heads: the two caches need no common strides."""
    c = Case(mxq, [333, 48, 1000], 3, 4, 256, False, page=48, seed=45)
    want = c.call()["out"]
    vq, vsf = empty_cache(c.vq.shape[0], 48, 3, 256, "hnd")
    vq.copy_(c.vq)
    vsf.copy_(c.vsf)
    c.vq, c.vsf = vq, vsf
    assert torch.equal(c.call()["out"], want)


def test_common_pages_within_a_sequence(mxq):  # noqa: F811
    """A table may name a page more than once."""
    c = Case(mxq, [512], 1, 16, 128, True, seed=46)
    c.table[0, 4:] = c.table[0, :4]
    fill(c.g, c.kq, c.ksf, c.table, c.lens, 116, 2)
    c.check(c.call())


FIRST_CALL = """
import torch
import mxfp8_activation_quant_gb300 as m
g = torch.Generator(device="cuda").manual_seed(1)
c = m.MXFP8Cache.empty(5, 16, 1, 256)
k = torch.randn((70, 1, 256), generator=g, device="cuda").to(torch.bfloat16)
q = torch.randn((1, 9, 256), generator=g, device="cuda").to(torch.bfloat16)
slots = torch.arange(70, dtype=torch.int32, device="cuda")
table, seq = torch.arange(5, dtype=torch.int32, device="cuda").view(1, 5), torch.full((1,), 70, dtype=torch.int32, device="cuda")
out, want = torch.zeros_like(q), torch.empty_like(q)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    m.kv_write_mxfp8(k, slots, c)
    m.paged_attention_mxfp8(q, c, table, seq, 0.0625, out=out)
graph.replay()
m.paged_attention_mxfp8(q, c, table, seq, 0.0625, out=want)
torch.cuda.synchronize()
assert torch.equal(out, want) and bool(out.any())
print("fine")
"""


def test_first_call_under_capture(mxq):  # noqa: F811
    """A process whose first calls are captured ones: nothing has to be set up by an eager call."""
    import os
    import subprocess
    import sys

    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "fine", r.stderr[-2000:]


@pytest.mark.parametrize("page", [16, 48, 64])
def test_pages_that_end_inside_a_tile(mxq, page):  # noqa: F811
    """Lengths around every multiple of 16 up to two tiles, one CTA's item next to another's, in 64 bits."""
    lens = [n + d for n in range(16, 272, 16) for d in (-1, 0, 1)]
    c = Case(mxq, lens, 1, 12, 384, False, page=page, seed=47)
    out = c.call()
    c.check(out)


def test_a_longer_table_changes_nothing(mxq):  # noqa: F811
    """Columns of the table behind a sequence's pages hold anything."""
    c = Case(mxq, [300, 64, 1], 2, 8, 128, False, page=16, seed=48)
    want = c.call()
    wide = torch.full((3, 1000), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    wide[:, ::2] = -(2 ** 31)
    wide[:, :c.table.shape[1]] = c.table
    for b, n in enumerate(c.lens):
        wide[b, -(-n // 16):] = 7 if b == 1 else -9
    c.table = wide
    got = c.call()
    assert torch.equal(got["out"], want["out"]) and torch.equal(got["lse"], want["lse"])


@pytest.mark.parametrize("B,kv,G,D,page", [(65536, 1, 1, 128, 16), (64, 1024, 4, 128, 16), (3, 1, 4096, 256, 32), (1, 1024, 1, 512, 64)])
def test_the_largest_batches_and_heads(mxq, B, kv, G, D, page):  # noqa: F811
    """The most sequences, cache heads and query heads that a call takes; some sequences are checked in 64 bits."""
    from kv_reference import attention

    g = torch.Generator(device="cuda").manual_seed(B + kv)
    pages = B + 1
    shape = (pages, page, kv, D)
    code = torch.randint(0, 254, shape, generator=g, device="cuda", dtype=torch.int16)
    kq = (code + (code >= 127)).to(torch.uint8)
    ksf = torch.randint(114, 119, (*shape[:3], D // 32), generator=g, device="cuda", dtype=torch.int16).to(torch.uint8)
    table = torch.randperm(pages, generator=g, device="cuda")[:B].to(torch.int32).view(B, 1)
    seq = torch.randint(0, page + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    seq[0] = page
    q = torch.randn((B, kv * G, D), generator=g, device="cuda").to(torch.bfloat16)
    out, lse, scale = torch.full_like(q, math.nan), torch.empty((B, kv * G), device="cuda"), 2.0 / (math.sqrt(D) * 70 * 2.0 ** -11)
    mxq.paged_attention_mxfp8(q, mxq.MXFP8Cache(kq, ksf), table, seq, scale, out=out, lse=lse)
    pick = sorted({0, B // 3, B // 2, B - 1})
    o, l, tol, ltol = attention(q[pick], kq, ksf, None, None, table[pick], seq[pick].tolist(), scale)
    got = out[pick].double()
    assert bool(((got - o).abs() <= tol + 2.0 ** -8 * (o.abs() + tol) + 2.0 ** -133).all())
    assert bool((torch.where(l.isinf(), 0.0, (lse[pick].double() - l).abs()) <= ltol).all())
    assert torch.equal(lse.isinf(), (seq == 0)[:, None].expand_as(lse)) and not bool(out.isnan().any())


@pytest.mark.parametrize("G,D", [(8, 384), (8, 512), (16, 256), (12, 384), (16, 512), (32, 256), (64, 512)])
def test_values_of_their_own_at_length(mxq, G, D):  # noqa: F811
    """Rings of keys and values apart, long enough that loads overtake one another: a value cache that holds what the keys do gives
    what a latent call gives, but for the order of its sums (checked in 64 bits)."""
    g = torch.Generator(device="cuda").manual_seed(D + G)
    lens = [1 + (2711 * i) % 1500 for i in range(24)] + [1 + i for i in range(60)]
    c = Case(mxq, lens, 2, G, D, False, page=64, seed=50)
    c.vq.copy_(c.kq)
    c.vsf.copy_(c.ksf)
    out = c.call()
    c.vq = c.vsf = None
    want = c.call()
    err = (out["out"].double() - want["out"].double()).norm() / want["out"].double().norm()
    assert float(err) <= 2.0 ** -8 and not bool(out["out"].isnan().any())
    pick = torch.randint(0, len(lens), (6,), generator=g, device="cuda").tolist()
    c.q, c.table, c.lens = c.q[pick], c.table[pick], [lens[i] for i in pick]
    c.check(dict(out=out["out"][pick], lse=out["lse"][pick]))


def test_streams_by_object_and_by_handle(mxq):  # noqa: F811
    """stream= as a Stream, as a raw handle and as the default stream's 0; each has a workspace that grows."""
    small, large = Case(mxq, [40], 1, 8, 128, True, seed=51), two_cases(mxq)[1]
    want = [c.call()["out"] for c in (small, large)]
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream, 0, torch.cuda.default_stream()):
        for c, w in zip((small, large, small), (*want, want[0])):
            k, v = c.caches()
            out = torch.empty_like(c.q)
            torch.cuda.synchronize()
            mxq.paged_attention_mxfp8(c.q, k, c.table, c.seq, c.scale, v_cache=v, out=out, stream=stream)
            torch.cuda.synchronize()
            assert torch.equal(out, w)

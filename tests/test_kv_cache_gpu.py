"""kv_write_mxfp8 and kv_read_bf16: bytes and scales of mxfp8_quantize in their slots and nothing else touched;
rows read back as the values that the bytes stand for."""
import pytest
import torch

from kv_reference import empty_cache, fill, pages_for, values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mxq():
    from mxfp8_activation_quant_gb300 import build

    build.build()
    import mxfp8_activation_quant_gb300 as m

    assert torch.cuda.is_available(), "GPU tests need CUDA"
    m.load()
    return m


def rows(gen, T, heads, D, stride=None):
    """bf16 rows of widely spread magnitudes, zeros among them; stride: tokens that far apart."""
    x = torch.randn((T, heads, D), generator=gen, device="cuda") * torch.exp(3 * torch.randn((T, heads, D // 32, 1), generator=gen, device="cuda")).expand(-1, -1, -1, 32).reshape(T, heads, D)
    x[torch.rand((T, heads, D), generator=gen, device="cuda") < 0.1] = 0
    x = x.to(torch.bfloat16)
    if stride is None:
        return x
    wide = torch.full((T, stride), float("nan"), dtype=torch.bfloat16, device="cuda")
    out = wide[:, :heads * D].view(T, heads, D)
    out.copy_(x)
    return out


def quantized(mxq, x):
    """mxfp8_quantize of every row."""
    T, heads, D = x.shape
    q, sf = mxq.quantize(x.contiguous().view(T * heads, D), layouts=(mxq.SF_ROWMAJOR_U8,))
    return q.view(T, heads, D), sf[mxq.SF_ROWMAJOR_U8].view(T, heads, D // 32)


@pytest.mark.parametrize("T,heads,D,page,order,latent", [
    (1, 1, 512, 64, "nhd", True), (3, 1, 384, 16, "hnd", True), (1, 8, 128, 16, "hnd", False), (100, 8, 128, 64, "nhd", False),
    (37, 3, 96, 48, "hnd", False), (129, 5, 32, 1, "nhd", False), (70, 2, 1024, 7, "hnd", False), (515, 16, 192, 80, "nhd", True),
])
def test_write(mxq, T, heads, D, page, order, latent):
    g = torch.Generator(device="cuda").manual_seed(T + D)
    pages = -(-T // page) + 2
    tensors = []
    for i in range(1 if latent else 2):
        hd, dd = (heads, D) if i == 0 else (heads + 1, D)  # the values' heads may be others
        q, sf = empty_cache(pages, page, hd, dd, order, pad=i)
        tensors.append((rows(g, T, hd, dd, None if i == 0 else hd * dd + 64), mxq.MXFP8Cache(q, sf)))
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:T].to(torch.int32)
    slots[::7] = torch.tensor([-1, pages * page, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device="cuda").repeat(T)[:len(slots[::7])]
    want = []
    for x, c in tensors:
        q, e = quantized(mxq, x)
        base = c.data._base.clone(), c.sf._base.clone()
        wq, ws = base[0].as_strided(c.data.shape, c.data.stride()), base[1].as_strided(c.sf.shape, c.sf.stride())
        for t, s in enumerate(slots.tolist()):
            if 0 <= s < pages * page:
                wq[s // page, s % page], ws[s // page, s % page] = q[t], e[t]
        want.append(base)
    args = () if latent else tensors[1]
    mxq.kv_write_mxfp8(tensors[0][0], slots, tensors[0][1], *args)
    for (x, c), (wq, ws) in zip(tensors, want):
        assert torch.equal(c.data._base, wq) and torch.equal(c.sf._base, ws)


def test_write_past_32_bits(mxq):
    """Slots whose rows lie more than 2^32 bytes into the cache."""
    pages, page, D = 70000, 128, 512
    q = torch.empty((pages, page, 1, D), dtype=torch.uint8, device="cuda")
    sf = torch.empty((pages, page, 1, D // 32), dtype=torch.uint8, device="cuda")
    c = mxq.MXFP8Cache(q, sf)
    g = torch.Generator(device="cuda").manual_seed(0)
    x = rows(g, 3, 1, D)
    slots = torch.tensor([pages * page - 1, 5, 69990 * page + 3], dtype=torch.int32, device="cuda")
    mxq.kv_write_mxfp8(x, slots, c)
    wq, ws = quantized(mxq, x)
    out = torch.empty((3, 1, D), dtype=torch.bfloat16, device="cuda")
    for t, s in enumerate(slots.tolist()):
        assert torch.equal(q[s // page, s % page], wq[t]) and torch.equal(sf[s // page, s % page], ws[t])
    table = torch.tensor([[pages - 1], [0], [69990]], dtype=torch.int32, device="cuda")
    starts = torch.tensor([page - 1, 5, 3], dtype=torch.int32, device="cuda")
    mxq.kv_read_bf16(c, table, torch.arange(4, dtype=torch.int32, device="cuda"), out, starts=starts)
    assert torch.equal(out.double(), values(wq, ws).to(torch.bfloat16).double())


@pytest.mark.parametrize("lens,heads,D,page,order,latent", [
    ([1], 1, 512, 64, "nhd", True), ([0, 5, 0, 0, 130, 1], 3, 96, 48, "hnd", False), ([333], 2, 384, 16, "hnd", True),
    ([17] * 40 + [0] * 30 + [64] * 5, 1, 32, 1, "nhd", False), (list(range(1100)), 1, 128, 100, "hnd", True),
])
def test_read(mxq, lens, heads, D, page, order, latent):
    g = torch.Generator(device="cuda").manual_seed(sum(lens) + D)
    B = len(lens)
    start = torch.randint(0, 20, (B,), generator=g, device="cuda").to(torch.int32)
    ends = [n + int(s) for n, s in zip(lens, start)]
    table, pages = pages_for(g, ends, page)
    table[B // 2, 0] = pages  # a page outside the cache: zeros
    table[B - 1, -1] = -1
    front, behind = 3, 5      # rows in front of the first and behind the last sequence
    cu = torch.full((B + 1,), front, dtype=torch.int32, device="cuda")
    cu[1:] += torch.tensor(lens, dtype=torch.int32, device="cuda").cumsum(0).to(torch.int32)
    total = front + sum(lens) + behind
    caches, outs = [], []
    for i in range(1 if latent else 2):
        q, sf = empty_cache(pages, page, heads, D, order, pad=i)
        fill(g, q, sf, table, ends, mean=127, spread=100)
        caches.append(mxq.MXFP8Cache(q, sf))
        outs.append(torch.full((total, heads, D), 7.0, dtype=torch.bfloat16, device="cuda"))
    mxq.kv_read_bf16(caches[0], table, cu, outs[0], *((caches[1], outs[1]) if not latent else ()), starts=start)
    for c, out in zip(caches, outs):
        want = torch.full((total, heads, D), 7.0, dtype=torch.float64, device="cuda")
        for b, n in enumerate(lens):
            if n:
                pos = torch.arange(n, device="cuda") + start[b]
                p = table[b].long()[pos // page]
                ok = (p >= 0) & (p < pages)
                v = values(c.data[p.clamp(0, pages - 1), pos % page], c.sf[p.clamp(0, pages - 1), pos % page])
                want[int(cu[b]):int(cu[b + 1])] = torch.where(ok[:, None, None], v, 0.0)
        # (through fp32, which holds every product of a code and a scale down to 2^-136)
        assert torch.equal(out, want.float().to(torch.bfloat16))


def test_read_without_starts_and_behind_the_table(mxq):
    """Positions past the table's width read as zeros."""
    g = torch.Generator(device="cuda").manual_seed(3)
    q, sf = empty_cache(4, 16, 1, 128)
    table = torch.tensor([[2, 0]], dtype=torch.int32, device="cuda")
    fill(g, q, sf, table, [32])
    out = torch.full((40, 1, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    mxq.kv_read_bf16(mxq.MXFP8Cache(q, sf), table, torch.tensor([0, 40], dtype=torch.int32, device="cuda"), out)
    v = values(torch.cat([q[2], q[0]]), torch.cat([sf[2], sf[0]])).to(torch.bfloat16)
    assert torch.equal(out[:32], v) and not out[32:].any()


def test_write_then_read_is_the_quantized_value(mxq):
    """Exhaustive: every finite bf16 alone in its group, through the cache and back."""
    x = torch.arange(0, 1 << 16, device="cuda").to(torch.int32).to(torch.int16).view(torch.bfloat16)
    x = torch.where(torch.isfinite(x), x, 0.0)
    rows_ = torch.zeros((1 << 14, 4, 32), dtype=torch.bfloat16, device="cuda")
    rows_[:, :, 5] = x.view(-1, 4)
    rows_ = rows_.view(1 << 14, 1, 128)
    q, sf = empty_cache(1 << 8, 64, 1, 128)
    c = mxq.MXFP8Cache(q, sf)
    mxq.kv_write_mxfp8(rows_, torch.arange(1 << 14, dtype=torch.int32, device="cuda"), c)
    out = torch.empty_like(rows_)
    table = torch.arange(1 << 8, dtype=torch.int32, device="cuda").view(1, -1)
    mxq.kv_read_bf16(c, table, torch.tensor([0, 1 << 14], dtype=torch.int32, device="cuda"), out)
    wq, ws = quantized(mxq, rows_)
    assert torch.equal(q.reshape(wq.shape), wq) and torch.equal(sf.reshape(ws.shape), ws)
    assert torch.equal(out, values(wq, ws).float().to(torch.bfloat16))
    # From 248 * 2^120 on the nearest code is 256 with the scale 2^120: the value 2^128, which bf16 has as infinity.
    x = rows_.double()
    top = x.abs() >= 248 * 2.0 ** 120
    assert torch.equal(out.isinf(), top) and int(top.sum()) == 16  # (8 mantissas, 2 signs)
    err = torch.where(top, 0.0, (out.double() - x).abs())
    assert bool((err <= 2.0 ** -4 * x.abs() + 2.0 ** -137).all())


def test_captured(mxq):
    """A write and a read in one CUDA graph, replayed with other tokens and slots."""
    g = torch.Generator(device="cuda").manual_seed(9)
    q, sf = empty_cache(6, 16, 2, 128)
    c = mxq.MXFP8Cache(q, sf)
    x, slots = rows(g, 5, 2, 128), torch.arange(5, dtype=torch.int32, device="cuda")
    out = torch.empty_like(x)
    table, cu = torch.zeros((5, 1), dtype=torch.int32, device="cuda"), torch.arange(6, dtype=torch.int32, device="cuda")
    starts = torch.zeros(5, dtype=torch.int32, device="cuda")

    def step():
        mxq.kv_write_mxfp8(x, slots, c)
        mxq.kv_read_bf16(c, table, cu, out, starts=starts)

    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        step()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3):
        x.copy_(rows(g, 5, 2, 128))
        slots.copy_(torch.randperm(96, generator=g, device="cuda")[:5])
        table.copy_((slots // 16).view(5, 1))
        starts.copy_(slots % 16)
        graph.replay()
        assert torch.equal(out, values(*quantized(mxq, x)).float().to(torch.bfloat16))


@pytest.mark.parametrize("T,heads,dim,two", [(32769, 1, 512, False), (16387, 5, 160, True), (33000, 1, 32, True)])
def test_many_tokens(mxq, T, heads, dim, two):
    """Numbers of warps and slots past 2^15, some tokens not written, values of another width."""
    g = torch.Generator(device="cuda").manual_seed(T)
    pages = -(-T // 16) + 2
    slots = torch.randperm(pages * 16, generator=g, device="cuda")[:T].to(torch.int32)
    slots[torch.rand(T, generator=g, device="cuda") < 0.2] = -1
    slots[T - 3:] = torch.tensor([-1, pages * 16, -(2 ** 31)], dtype=torch.int32)
    pairs = [(rows(g, T, heads, dim), empty_cache(pages, 16, heads, dim))]
    if two:
        pairs.append((rows(g, T, 2, 64), empty_cache(pages, 16, 2, 64)))
    caches = [mxq.MXFP8Cache(*c) for _, c in pairs]
    mxq.kv_write_mxfp8(pairs[0][0], slots, caches[0], pairs[1][0] if two else None, caches[1] if two else None)
    ok = (slots >= 0) & (slots < pages * 16)
    for x, (q, sf) in pairs:
        wq, ws = quantized(mxq, x)
        want, wsf = torch.full_like(q, 0x7F), torch.full_like(sf, 0xFF)
        want.view(-1, *q.shape[2:])[slots[ok].long()] = wq.view(x.shape)[ok]
        wsf.view(-1, *sf.shape[2:])[slots[ok].long()] = ws.view(*x.shape[:2], -1)[ok]
        assert torch.equal(q, want) and torch.equal(sf, wsf)

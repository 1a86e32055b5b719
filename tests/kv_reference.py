"""Paged MXFP8 caches for tests and their operators in 64 bits, from the definitions."""
import torch


def values(q, sf):
    """fp64 values of E4M3 bytes [.., D] with UE8M0 bytes [.., D / 32]."""
    scale = torch.where(sf == 0, 2.0 ** -127, ((sf.long() + 896) << 52).view(torch.float64))
    return q.view(torch.float8_e4m3fn).double() * scale.repeat_interleave(32, dim=-1)


def empty_cache(pages, page, heads, D, order="nhd", pad=0, device="cuda"):
    """Bytes and scales [pages, page, heads, ..]; "hnd" keeps a head's tokens together; pad: rows of other data
    between the pages. All of it NaN: what nobody writes must not matter."""
    shape = (page + pad, heads) if order == "nhd" else (heads, page + pad)
    q = torch.full((pages, *shape, D), 0x7F, dtype=torch.uint8, device=device)
    sf = torch.full((pages, *shape, D // 32), 0xFF, dtype=torch.uint8, device=device)
    if order == "hnd":
        q, sf = q.transpose(1, 2), sf.transpose(1, 2)
    return q[:, :page], sf[:, :page]


def fill(gen, q, sf, table, lens, mean=118, spread=3):
    """Random bytes (no NaN codes) and scales around `mean` for the tokens that the table and lens name."""
    page = q.shape[1]
    for b, n in enumerate(lens):
        for j in range(min(-(-n // page), table.shape[1])):
            p, m = int(table[b, j]), min(page, n - j * page)
            if not 0 <= p < q.shape[0]:
                continue
            code = torch.randint(0, 254, (m, *q.shape[2:]), generator=gen, device=q.device)
            q[p, :m] = (code + (code >= 127)).to(torch.uint8)  # 0..126, 128..254
            sf[p, :m] = torch.randint(mean - spread, mean + spread + 1, (m, *sf.shape[2:]), generator=gen,
                                      device=q.device).to(torch.uint8)


def pages_for(gen, lens, page, spare=2, width=None, device="cuda"):
    """A table of distinct pages in random order, and the number of pages."""
    width = width or max(1, max(-(-max(n, 0) // page) for n in lens))
    n = len(lens) * width
    order = torch.randperm(n + spare, generator=gen, device=device)[:n]
    return order.to(torch.int32).view(len(lens), width).contiguous(), n + spare


def attention(qt, kq, ksf, vq, vsf, table, lens, scale, p_bits=2.0 ** -11):
    """o, lse in fp64 and how far a result may be off before its rounding to bf16:
    - the score: q as two MXFP8 numbers (2^-21 of the group's largest magnitude), D products added in fp32
      (each of at most 2 D + 2 roundings of 2^-24 of the sum of magnitudes), scale and base change (2^-22 of it)
    - a probability: e^score's error, p_bits for its 16 bits, 2^-20 for the exponential, and below the
      smallest normal fp16 (against the largest, 1) 2^-25 absolute
    - sums in fp32 over n tokens: a rounding of 2^-24 for every 16 of them, and one per split
    """
    B, H, D = qt.shape
    kv, page, pages = kq.shape[2], kq.shape[1], kq.shape[0]
    G = H // kv
    o = torch.zeros((B, H, D), dtype=torch.float64, device=qt.device)
    lse = torch.full((B, H), -float("inf"), dtype=torch.float64, device=qt.device)
    tol, ltol = torch.zeros_like(o), torch.zeros((B, H), dtype=torch.float64, device=qt.device)
    for b, n in enumerate(lens):
        n = min(int(n), table.shape[1] * page)
        if n <= 0:
            continue
        pos = torch.arange(n, device=qt.device)
        p = table[b].long()[pos // page]
        ok = (p >= 0) & (p < pages)
        p, at = p[ok], (pos % page)[ok]
        if not p.numel():
            continue
        k = values(kq[p, at], ksf[p, at])
        v = k if vq is None else values(vq[p, at], vsf[p, at])
        for h in range(kv):
            q = qt[b, h * G:(h + 1) * G].double()
            s = scale * (q @ k[:, h].T)
            qg = q.abs().view(G, D // 32, 32).amax(2).repeat_interleave(32, dim=1)
            kk = k[:, h].abs().T
            ds = abs(scale) * (2.0 ** -21 * (qg @ kk) + 2.0 ** -24 * (2 * D + 2) * (q.abs() @ kk)) + 2.0 ** -22 * s.abs()
            m = s.amax(1, keepdim=True)
            e = torch.exp(s - m)
            l = e.sum(1, keepdim=True)
            pr = e / l
            va = v[:, h].abs()
            o[b, h * G:(h + 1) * G] = pr @ v[:, h]
            lse[b, h * G:(h + 1) * G] = (m + torch.log(l))[:, 0]
            # l's own error is the mean of e's, so it counts once more for the whole sum
            rel = torch.expm1(ds) + p_bits + 2.0 ** -20 + 2.0 ** -24 * (n / 16 + 256)
            mean_rel = (pr * rel).sum(1, keepdim=True)
            tol[b, h * G:(h + 1) * G] = (pr * rel) @ va + mean_rel * (pr @ va) + 2.0 ** -25 / l * va.sum(0)
            ltol[b, h * G:(h + 1) * G] = (mean_rel[:, 0] - p_bits) + 2.0 ** -23 * (lse[b, h * G:(h + 1) * G].abs() + 1)
    return o, lse, tol, ltol

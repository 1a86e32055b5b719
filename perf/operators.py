"""Cases and plain forms of the mixture-of-experts half of a decoder layer: the residual's addition
with RMSNorm and MXFP8 output, the routing to experts, and the experts' products in MXFP8.

``run`` is the plain form (elementary torch operations in 32 bits, 64 where a choice between near
values depends on them) or, with ``own`` set, the calls a user makes of the framework.
"""
import math

import torch

own = False

E4M3_MAX = 448.0


# ---- cases -----------------------------------------------------------------------------------
def listed():
    return [
        # one decoded token of one sequence: latency is all that counts
        dict(name="norm 1 token", op="norm", T=1, H=5120, stream="bf16", sf="rowmajor"),
        # a ragged chunk of a prompt, with the residual stream kept in fp32, at another width
        dict(name="norm 333 fp32 stream", op="norm", T=333, H=7168, stream="fp32", sf="rowmajor"),
        # a full prefill step feeding an MXFP8 GEMM (the tensor cores' scale layout)
        dict(name="norm 8192 tokens", op="norm", T=8192, H=5120, stream="bf16", sf="tiled"),
        # one decoded token, 256 experts in 8 groups of which 4 are kept, balance bias
        dict(name="route 1 token", op="route", T=1, E=256, k=8, dtype="fp32", scoring="sigmoid", bias=True,
             groups=8, kept=4, top=2, renorm=True, scale=2.5, masked=0.0),
        # a ragged chunk through a softmax router with bf16 logits, some experts switched off
        dict(name="route 1001 softmax", op="route", T=1001, E=160, k=6, dtype="bf16", scoring="softmax", bias=False,
             groups=8, kept=3, top=1, renorm=False, scale=1.0, masked=0.05),
        # a long prefill step of the grouped sigmoid router
        dict(name="route 16384 tokens", op="route", T=16384, E=256, k=8, dtype="fp32", scoring="sigmoid", bias=True,
             groups=8, kept=4, top=2, renorm=True, scale=2.5, masked=0.0),
        # one decoded token through 8 of 64 experts: the weights of 8 experts stream once
        dict(name="experts 1 token", op="experts", T=1, E=64, k=8, H=5120, I=1024, idle=0.0, x_sf="rowmajor"),
        # a decode batch padded to its graph's size: a quarter of the slots route nowhere
        dict(name="experts 48 tokens", op="experts", T=48, E=64, k=8, H=5120, I=1024, idle=0.25, x_sf="rowmajor"),
        # an odd chunk through a small model with few experts
        dict(name="experts 333 small", op="experts", T=333, E=40, k=3, H=2048, I=640, idle=0.0, x_sf="tiled"),
        # a prompt chunk that reaches every expert with a ragged number of tokens
        dict(name="experts 777 tokens", op="experts", T=777, E=64, k=8, H=5120, I=1024, idle=0.0, x_sf="rowmajor"),
        # a full prefill step
        dict(name="experts 4096 tokens", op="experts", T=4096, E=64, k=8, H=5120, I=1024, idle=0.0, x_sf="rowmajor"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "route", "experts"])
    if op == "norm":
        sf = rng.choice(["rowmajor", "tiled", "packed"])
        step = 128 if sf == "packed" else 32
        H = (min(8192 // step - 1, _log_int(rng, 512, 8192) // step) | 1) * step
        T = _log_int(rng, 1, 8192)
        T = max(1, min(T, 8192 * 5120 * 9 // (H * 13)))
        return dict(op=op, T=T, H=H, stream=rng.choice(["bf16", "bf16", "fp32"]), sf=sf)
    if op == "route":
        groups = rng.choice([1, 1, 4, 8])
        E = groups * rng.randint(4, 64 if groups < 8 else 32)
        kept = rng.randint(1, groups)
        k = rng.randint(1, min(16, kept * (E // groups)))
        T = min(_log_int(rng, 1, 16384), 16384 * 256 // E)
        return dict(op=op, T=T, E=E, k=k, dtype=rng.choice(["fp32", "bf16"]), scoring=rng.choice(["sigmoid", "softmax"]),
                    bias=rng.random() < 0.5, groups=groups, kept=kept, top=rng.choice([1, 2]),
                    renorm=rng.random() < 0.5, scale=rng.choice([1.0, 2.5]), masked=rng.choice([0.0, 0.0, 0.1]))
    H = rng.choice([512, 768, 1024, 1280, 1536, 2048, 2176, 2560, 2944, 3584, 4096, 4992, 5120, 6144])
    I = 128 * rng.randint(2, 11)
    E = min(_log_int(rng, 8, 128), 64 * 5120 * 1024 // (H * I))
    E = max(E, 4)
    k = rng.randint(1, min(8, E))
    T = _log_int(rng, 1, 4096)
    T = max(1, min(T, 4096 * 8 * 5120 * 1024 // (H * I * k)))
    return dict(op=op, T=T, E=E, k=k, H=H, I=I, idle=rng.choice([0.0, 0.0, 0.25]), x_sf=rng.choice(["rowmajor", "tiled"]))


def work(case):
    c = case
    if c["op"] == "norm":
        s = 2 if c["stream"] == "bf16" else 4
        n = c["T"] * c["H"]
        return {"bytes": n * (2 + 2 * s + 2 + 1 + 1 / 32) + 2 * c["H"], "flops": 6 * n}
    if c["op"] == "route":
        b = 2 if c["dtype"] == "bf16" else 4
        return {"bytes": c["T"] * (c["E"] * b + c["k"] * 8) + (4 * c["E"] if c["bias"] else 0),
                "flops": 8 * c["T"] * c["E"]}
    pairs = c["T"] * c["k"] * (1 - c["idle"])
    active = c["E"] * (1 - (1 - c["k"] / c["E"]) ** (c["T"] * (1 - c["idle"])))
    weights = active * 3 * c["H"] * c["I"] * 33 / 32
    return {"bytes": weights + c["T"] * c["H"] * (33 / 32 + 2) + c["T"] * c["k"] * 8,
            "flops": pairs * 6 * c["H"] * c["I"]}


# ---- inputs ----------------------------------------------------------------------------------
def _pow2(e):
    """2^e in fp32 for whole e in [-126, 127], from the bits (a device's exp2 need not be exact)."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _quantize(x, group=32):
    """fp32 [..., K] -> E4M3 values (torch.float8_e4m3fn), UE8M0 bytes [..., K/32]: the smallest
    power-of-two scale that brings the group's largest magnitude to 448 or below."""
    g = x.view(*x.shape[:-1], x.shape[-1] // group, group)
    m, e = torch.frexp(g.abs().amax(-1).clamp_min(2.0 ** -126))  # amax = m 2^e, m in [0.5, 1)
    e = (e - 9 + (m > 0.875).to(e.dtype) + 127).clamp_min(0)     # 448 = 0.875 * 2^9
    q = (g * _pow2(127 - e)[..., None]).to(torch.float8_e4m3fn)
    return q.view(x.shape), e.to(torch.uint8)


def _tile_scales(sf):
    """Row-major UE8M0 bytes [M, G] -> the tensor cores' F8_128x4 layout, flat."""
    M, G = sf.shape
    Mp, Gp = -(-M // 128) * 128, -(-G // 4) * 4
    p = torch.zeros((Mp, Gp), dtype=torch.uint8, device=sf.device)
    p[:M, :G] = sf
    return p.view(Mp // 128, 4, 32, Gp // 4, 4).permute(0, 3, 2, 1, 4).reshape(-1).contiguous()


def _pack_scales(sf):
    """Row-major UE8M0 bytes [M, G] -> int32 words of four groups, rows contiguous, flat bytes."""
    M, G = sf.shape
    Mp = -(-M // 4) * 4
    p = torch.zeros((Mp, G), dtype=torch.uint8, device=sf.device)
    p[:M] = sf
    return p.view(Mp, G // 4, 4).permute(1, 0, 2).reshape(-1).contiguous()


def _weights(gen, experts, rows, cols):
    """MXFP8 weights of all experts, N(0, 1/sqrt(cols)): E4M3 bytes, row-major and tiled scales."""
    q = torch.empty((experts * rows, cols), dtype=torch.uint8, device="cuda")
    sf = torch.empty((experts * rows, cols // 32), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 27) // (rows * cols)) * rows
    for r in range(0, experts * rows, step):
        n = min(step, experts * rows - r)
        w = torch.randn((n, cols), generator=gen, device="cuda").mul_(cols ** -0.5)
        v, s = _quantize(w)
        q[r:r + n] = v.view(torch.uint8)
        sf[r:r + n] = s
    return dict(q=q, sf=sf, tiled=_tile_scales(sf))


def _stream_input(gen, T, H):
    """Activations with a few large channels, as a residual stream has them."""
    x = torch.randn((T, H), generator=gen, device="cuda")
    big = torch.randint(0, H, (max(1, H // 1000),), generator=gen, device="cuda")
    x[:, big] *= 30.0
    return x


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    T = c["T"]
    if c["op"] == "norm":
        st = torch.bfloat16 if c["stream"] == "bf16" else torch.float32
        x = torch.randn((T, c["H"]), generator=gen, device="cuda").to(torch.bfloat16)
        residual = (_stream_input(gen, T, c["H"]) * 3.0).to(st)
        gamma = (1.0 + 0.1 * torch.randn(c["H"], generator=gen, device="cuda")).to(torch.bfloat16)
        return dict(c, x=x, residual=residual, gamma=gamma, eps=1e-6)
    if c["op"] == "route":
        E = c["E"]
        logits = 1.5 * torch.randn((T, E), generator=gen, device="cuda") + 0.5 * torch.randn(E, generator=gen, device="cuda")
        logits = logits.to(torch.float32 if c["dtype"] == "fp32" else torch.bfloat16)
        if c["masked"]:
            off = torch.rand((T, E), generator=gen, device="cuda") < c["masked"]
            logits.masked_fill_(off, -math.inf)
        bias = 0.1 * torch.randn(E, generator=gen, device="cuda") if c["bias"] else None
        return dict(c, logits=logits, bias_t=bias)
    E, k, H, I = c["E"], c["k"], c["H"], c["I"]
    x = _stream_input(gen, T, H)
    xq, xsf = _quantize(x.to(torch.bfloat16).float())
    pop = torch.randn((T, E), generator=gen, device="cuda") + 0.4 * torch.randn(E, generator=gen, device="cuda")
    top = torch.topk(pop, k, dim=1)
    ids = top.indices.to(torch.int32)
    w = torch.softmax(top.values, dim=1).to(torch.float32)
    if c["idle"]:
        n = int(T * c["idle"])
        if n:
            ids[T - n:] = -1  # padding tokens of a fixed-size batch
    return dict(c, xq=xq.view(torch.uint8), xsf=xsf, xtiled=_tile_scales(xsf), ids=ids.contiguous(), w=w.contiguous(),
                w13=_weights(gen, E, 2 * I, H), w2=_weights(gen, E, H, I))


# ---- plain forms -----------------------------------------------------------------------------
def _plain_norm(s):
    h = (s["x"].float() + s["residual"].float()).to(s["residual"].dtype)
    f = h.double()  # a value next to a rounding border decides its group's scale
    r = torch.rsqrt(f.square().mean(1, keepdim=True) + s["eps"])
    y = (f * r * s["gamma"].double()).to(torch.bfloat16)
    q, e = _quantize(y.float())
    sf = e if s["sf"] == "rowmajor" else _tile_scales(e) if s["sf"] == "tiled" else _pack_scales(e)
    return dict(residual=h, y=y, y_q=q, y_sf=sf.reshape(-1).view(torch.float8_e8m0fnu))


def _plain_route(s):
    l = s["logits"].double()
    T, E = l.shape
    k, G = s["k"], s["groups"]
    there = l > -math.inf
    if s["scoring"] == "sigmoid":
        score = torch.sigmoid(l)
    else:
        score = torch.softmax(l, dim=1)
    choice = score + s["bias_t"].double() if s["bias"] else score
    order = choice if s["bias"] else l
    choice = choice.masked_fill(~there, -math.inf)
    order = order.masked_fill(~there, -math.inf)
    if G > 1:
        best = choice.view(T, G, E // G).sort(dim=2, descending=True).values[:, :, :s["top"]]
        value = torch.where(best > -math.inf, best, 0.0).sum(2).masked_fill(best[:, :, 0] == -math.inf, -math.inf)
        kept = value.sort(dim=1, descending=True, stable=True).indices[:, :s["kept"]]
        keep = torch.zeros((T, G), dtype=torch.bool, device=l.device).scatter_(1, kept, True)
        order = order.masked_fill(~keep.repeat_interleave(E // G, dim=1), -math.inf)
    top = order.sort(dim=1, descending=True, stable=True)
    ids, found = top.indices[:, :k], top.values[:, :k] > -math.inf
    w = torch.where(found, score.gather(1, ids), 0.0)
    if s["renorm"]:
        w = w / (w.sum(1, keepdim=True) + 1e-20)
    return dict(ids=torch.where(found, ids, -1).to(torch.int32), weights=(w * s["scale"]).float())


def _dequantize(q, sf):
    v = q.view(torch.float8_e4m3fn).float()
    return (v.view(*q.shape[:-1], -1, 32) * sf.view(torch.float8_e8m0fnu).float()[..., None]).view(q.shape)


def _plain_experts(s):
    T, E, k, H, I = s["T"], s["E"], s["k"], s["H"], s["I"]
    x = _dequantize(s["xq"], s["xsf"])
    P = T * k
    # the (token, slot) pairs sorted by expert and cut into blocks of at most B pairs of one expert
    B = 1 if P <= 64 else 16 if P <= 4096 else 128
    blocks = -(-P // B) + min(E, P)
    ids = s["ids"].long().view(-1)
    valid = (ids >= 0) & (ids < E)
    key = torch.where(valid, ids, E)
    by = key.sort(stable=True)
    count = torch.zeros(E + 1, dtype=torch.long, device=x.device).scatter_add_(0, key, torch.ones_like(key))
    first = count.cumsum(0) - count
    nb = -(-count // B)
    nb[E:] = 0
    b0 = nb.cumsum(0) - nb
    rank = torch.arange(P, device=x.device) - first[by.values]
    slot = torch.where(by.values < E, (b0[by.values] + rank // B) * B + rank % B, blocks * B)
    token = torch.full((blocks * B + 1,), T, dtype=torch.long, device=x.device)
    token[slot] = by.indices // k
    expert = torch.zeros(blocks + 1, dtype=torch.long, device=x.device)
    expert[slot // B] = by.values.clamp(max=E - 1)
    token, expert = token[:-1].view(blocks, B), expert[:-1]
    xs = torch.cat([x, x.new_zeros(1, H)])[token]
    w13 = _dequantize(s["w13"]["q"].view(E, 2 * I, H)[expert], s["w13"]["sf"].view(E, 2 * I, H // 32)[expert])
    gu = torch.bmm(xs, w13.transpose(1, 2))
    del w13
    g, u = gu[..., 0::2], gu[..., 1::2]
    h = (g / (1.0 + torch.exp(-g)) * u).to(torch.bfloat16).float()
    hq, hsf = _quantize(h.contiguous())
    h = _dequantize(hq.view(torch.uint8), hsf)
    w2 = _dequantize(s["w2"]["q"].view(E, H, I)[expert], s["w2"]["sf"].view(E, H, I // 32)[expert])
    y = torch.bmm(h, w2.transpose(1, 2)).view(blocks * B, H)
    del w2
    y = torch.cat([y, y.new_zeros(1, H)])
    place = torch.empty_like(slot)
    place[by.indices] = slot
    w = torch.where(valid, s["w"].view(-1), 0.0)
    out = (y[place].view(T, k, H) * w.view(T, k, 1)).sum(1)
    return dict(out=out.to(torch.bfloat16))


def _plain(s):
    return {"norm": _plain_norm, "route": _plain_route, "experts": _plain_experts}[s["op"]](s)


# ---- the framework's calls -------------------------------------------------------------------
def _own(s):
    import mxfp8_activation_quant_gb300 as m

    dev = "cuda"
    if s["op"] == "norm":
        T, H = s["x"].shape
        h = torch.empty_like(s["residual"])
        y = torch.empty((T, H), dtype=torch.bfloat16, device=dev)
        yq = torch.empty((T, H), dtype=torch.uint8, device=dev)
        layout = {"rowmajor": m.SF_ROWMAJOR_U8, "tiled": m.SF_TILED_128X4, "packed": m.SF_PACKED_I32_MN}[s["sf"]]
        sf = m.empty_sf(layout, T, H, dev)
        m.add_rmsnorm_dual_out(s["x"], s["residual"], s["gamma"], s["eps"], h, y, yq,
                               **{{"rowmajor": "sf_rowmajor", "tiled": "sf_128x4", "packed": "sf_packed"}[s["sf"]]: sf})
        return dict(residual=h, y=y, y_q=yq.view(torch.float8_e4m3fn), y_sf=sf.view(torch.float8_e8m0fnu))
    if s["op"] == "route":
        ids = torch.empty((s["T"], s["k"]), dtype=torch.int32, device=dev)
        w = torch.empty((s["T"], s["k"]), dtype=torch.float32, device=dev)
        m.moe_route(s["logits"], ids, w, bias=s["bias_t"], scoring=s["scoring"], groups=s["groups"],
                    topk_groups=s["kept"], group_top=s["top"], renormalize=s["renorm"], scale=s["scale"])
        return dict(ids=ids, weights=w)
    out = torch.empty((s["T"], s["H"]), dtype=torch.bfloat16, device=dev)
    x = m.MXFP8(s["xq"], s["xsf"], m.SF_ROWMAJOR_U8) if s["x_sf"] == "rowmajor" else m.MXFP8(s["xq"], s["xtiled"])
    m.moe_experts_mxfp8(x, s["ids"], s["w"], m.MXFP8(s["w13"]["q"], s["w13"]["tiled"]),
                        m.MXFP8(s["w2"]["q"], s["w2"]["tiled"]), out)
    return dict(out=out)


def run(state):
    return _own(state) if own else _plain(state)


# ---- from the definitions, in 64 bits --------------------------------------------------------
def _exact_codes(v):
    """E4M3 values and scales of bf16-valued fp64 [M, K], straight from the format's definition: the
    scale is found by search over the exponents, the value by rounding to the grid of its binade."""
    M, K = v.shape
    g = v.view(M, K // 32, 32)
    amax = g.abs().amax(2)
    two = lambda n: ((n.long() + 1023) << 52).view(torch.float64)  # noqa: E731
    e = torch.ceil(torch.log2(amax.clamp_min(2.0 ** -140) / 448.0))
    e = torch.where(448.0 * two(e - 1) >= amax, e - 1, e)
    e = torch.where(448.0 * two(e) < amax, e + 1, e).clamp_min(-127)
    z = g * two(-e)[..., None]
    binade = torch.floor(torch.log2(z.abs().clamp_min(2.0 ** -6)))
    binade = torch.where(two(binade) > z.abs().clamp_min(2.0 ** -6), binade - 1, binade)
    step = two(binade - 3)
    q = torch.round(z / step) * step  # ties to even
    return q.view(M, K), two(e)


def _bf16(v):
    return v.to(torch.bfloat16).double()


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "norm":
        h = s["x"].double() + s["residual"].double()
        h = h.to(s["residual"].dtype).double()
        y = h / torch.sqrt((h * h).sum(1, keepdim=True) / s["H"] + s["eps"]) * s["gamma"].double()
        q, sc = _exact_codes(_bf16(y))
        T, Gk = sc.shape
        if s["sf"] == "rowmajor":
            sf = sc.reshape(-1)
        else:
            rows = torch.arange(-(-T // 128) * 128 if s["sf"] == "tiled" else -(-T // 4) * 4, device=q.device)
            groups = torch.arange(-(-Gk // 4) * 4, device=q.device)
            r, c = rows[:, None], groups[None, :]
            if s["sf"] == "tiled":
                at = ((r // 128) * (groups.numel() // 4) + c // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + c % 4
            else:
                at = (c // 4 * rows.numel() + r) * 4 + c % 4
            sf = torch.full((rows.numel() * groups.numel(),), 2.0 ** -127, dtype=torch.float64, device=q.device)
            sf[at[:T, :Gk].reshape(-1)] = sc.reshape(-1)
        return dict(residual=h, y=y, y_q=q, y_sf=sf)
    if s["op"] == "route":
        l = s["logits"].double()
        T, E = l.shape
        e = torch.exp(l - (l.amax(1, keepdim=True) if s["scoring"] == "softmax" else 0.0))
        score = e / e.sum(1, keepdim=True) if s["scoring"] == "softmax" else e / (1 + e)
        c = score + (s["bias_t"].double() if s["bias"] else 0.0)
        c = torch.where(l == -math.inf, -math.inf, c)
        left = c.clone()
        if s["groups"] > 1:
            v, value = c.view(T, s["groups"], -1).clone(), None
            for _ in range(s["top"]):
                m = v.max(2)
                add = torch.where(m.values == -math.inf, 0.0, m.values)
                value = m.values if value is None else value + add
                v.scatter_(2, m.indices[..., None], -math.inf)
            ban = torch.ones((T, s["groups"]), dtype=torch.bool, device=l.device)
            for _ in range(s["kept"]):
                i = value.argmax(1, keepdim=True)
                ban.scatter_(1, i, False)
                value.scatter_(1, i, -math.inf)
            left = left.view(T, s["groups"], -1).masked_fill(ban[..., None], -math.inf).view(T, E)
        ws = []
        for _ in range(s["k"]):
            i = left.argmax(1, keepdim=True)
            ws.append(torch.where(left.gather(1, i) == -math.inf, 0.0, score.gather(1, i)))
            left.scatter_(1, i, -math.inf)
        w = torch.cat(ws, 1)
        if s["renorm"]:
            w = w / (w.sum(1, keepdim=True) + 1e-20)
        return dict(ids=None, weights=w * s["scale"])
    T, E, k, H, I = s["T"], s["E"], s["k"], s["H"], s["I"]

    def values(q, sf):
        scale = ((sf.long() + 896) << 52).view(torch.float64)
        return q.view(torch.float8_e4m3fn).double() * scale.repeat_interleave(32, dim=-1)

    x = values(s["xq"], s["xsf"])
    out = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    for e in range(E):
        t, j = torch.nonzero(s["ids"] == e, as_tuple=True)
        if not t.numel():
            continue
        gu = x[t] @ values(s["w13"]["q"][e * 2 * I:(e + 1) * 2 * I], s["w13"]["sf"][e * 2 * I:(e + 1) * 2 * I]).T
        g, u = gu[:, 0::2], gu[:, 1::2]
        q, sc = _exact_codes(_bf16(g * torch.sigmoid(g) * u))
        h = q * sc.repeat_interleave(32, dim=1)
        y = h @ values(s["w2"]["q"][e * H:(e + 1) * H], s["w2"]["sf"][e * H:(e + 1) * H]).T
        out.index_add_(0, t, y * s["w"][t, j].double()[:, None])
    return dict(out=out)

"""The sum over a token's experts in moe_experts_mxfp8 is held in 32 bits: exact cases with whole numbers."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mxq():
    from mxfp8_activation_quant_gb300 import build

    build.build()
    import mxfp8_activation_quant_gb300 as m

    assert torch.cuda.is_available(), "GPU tests need CUDA"
    m.load()
    return m


@pytest.fixture(scope="module")
def pair(mxq):
    """Two experts whose products nearly cancel, of an odd number of 128-row tiles and more k-blocks than
    the stages in flight. A feature's activation is 64 x, x in {0, 1}; W2 is 1 but for a few -1 and 0, and
    its negative for the other expert but for a few zeros: y_0 and y_1 = 64 m with |m| up to 1024, eleven
    bits, and y_0 + y_1 = 64 n with |n| small. Every product and every fp32 sum of them is exact."""
    H, I = 1152, 1024
    g = torch.Generator(device="cuda").manual_seed(11)
    wg = torch.zeros((2, I, H), dtype=torch.bfloat16, device="cuda")
    wg[:, :, 0] = 64.0
    wu = torch.zeros_like(wg)
    pick = torch.randint(1, H, (1, I), generator=g, device="cuda").expand(2, I)
    wu.scatter_(2, pick[:, :, None], 1.0)
    u = torch.rand((H, I), generator=g, device="cuda")
    w = torch.where(u < 0.05, -1.0, torch.where(u < 0.1, 0.0, 1.0))
    off = torch.rand((H, I), generator=g, device="cuda") < 0.02
    w2 = torch.stack((w, torch.where(off, 0.0, -w)))
    mx = lambda t: mxq.MXFP8(*(lambda r: (r[0], r[1][2]))(  # noqa: E731
        mxq.quantize(t.to(torch.bfloat16).contiguous(), layouts=(2,))))
    return dict(H=H, I=I, gen=g, pick=pick[0], w2=w2, mx=mx, w13=mx(mxq.interleave_gate_up(wg, wu)), w2q=mx(w2.view(2 * H, I)))


# (333 tokens: more than 160 rows per expert, so rows are copied; fewer are read in place)
@pytest.mark.parametrize("T", [1, 7, 150, 333])
def test_products_that_cancel(mxq, pair, T):
    H, g = pair["H"], pair["gen"]
    x = (torch.rand((T, H), generator=g, device="cuda") < 0.9).float()
    x[:, 0] = 1.0
    a = 64.0 * x[:, pair["pick"]].double()
    y = torch.stack([a @ pair["w2"][e].double().T for e in range(2)], 1)
    # some values of every expert need more bits than bf16 has
    assert (y != y.to(torch.bfloat16).double()).any()
    ids = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda").repeat(T, 1)
    ids[1::2] = ids[1::2].flip(1)
    for w in (1.0, 0.25):
        out = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
        status = mxq.new_status()
        mxq.moe_experts_mxfp8(pair["mx"](x), ids, torch.full((T, 2), w, device="cuda"), pair["w13"], pair["w2q"], out,
                              status=status)
        mxq.check_status(status)
        assert torch.equal(out, (w * y.sum(1)).to(torch.bfloat16))


@pytest.mark.parametrize("T,k", [(5, 40), (40, 64)])
def test_many_slots(mxq, pair, T, k):
    """More slots than lanes of a warp; the sum over them is exact in fp32 (|sum| < 2^24 quarters)."""
    H, g = pair["H"], pair["gen"]
    x = (torch.rand((T, H), generator=g, device="cuda") < 0.9).float()
    x[:, 0] = 1.0
    a = 64.0 * x[:, pair["pick"]].double()
    y = torch.stack([a @ pair["w2"][e].double().T for e in range(2)], 1)
    ids = torch.randint(-1, 2, (T, k), generator=g, device="cuda", dtype=torch.int32)
    w = 0.25 * torch.randint(1, 4, (T, k), generator=g, device="cuda").float()
    out = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    mxq.moe_experts_mxfp8(pair["mx"](x), ids, w, pair["w13"], pair["w2q"], out)
    want = sum(torch.where(ids == e, w, 0.0).double().sum(1, keepdim=True) * y[:, e] for e in range(2))
    assert torch.equal(out, want.to(torch.bfloat16))


def test_many_items(mxq):
    """Forty experts, 17 and 14 k-blocks, several items for every pair of SMs: the rings of stages, scales and
    accumulators go round many times, and every value is exact."""
    E, H, I, T, k = 40, 2176, 1792, 700, 4
    g = torch.Generator(device="cuda").manual_seed(12)
    wg = torch.zeros((E, I, H), dtype=torch.bfloat16, device="cuda")
    wg[:, :, 0] = 64.0
    wu = torch.zeros_like(wg)
    pick = torch.randint(1, H, (E, I), generator=g, device="cuda")
    wu.scatter_(2, pick[:, :, None], 1.0)
    u = torch.rand((E, H, I), generator=g, device="cuda")
    w2 = torch.where(u < 0.1, -1.0, torch.where(u < 0.3, 0.0, 1.0)) * torch.where(torch.rand((E, H, 1), generator=g, device="cuda") < 0.5, -1.0, 1.0)
    x = (torch.rand((T, H), generator=g, device="cuda") < 0.9).float()
    x[:, 0] = 1.0
    ids = torch.rand((T, E), generator=g, device="cuda").topk(k, dim=1).indices.to(torch.int32)
    w = 0.25 * torch.randint(1, 5, (T, k), generator=g, device="cuda").float()
    mx = lambda t: mxq.MXFP8(*(lambda r: (r[0], r[1][2]))(  # noqa: E731
        mxq.quantize(t.to(torch.bfloat16).contiguous(), layouts=(2,))))
    out = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    status = mxq.new_status()
    mxq.moe_experts_mxfp8(mx(x), ids, w, mx(mxq.interleave_gate_up(wg, wu)), mx(w2.view(E * H, I)), out, status=status)
    mxq.check_status(status)
    want = torch.zeros((T, H), dtype=torch.float64, device="cuda")
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        want.index_add_(0, t, (64.0 * x[t][:, pick[e]].double()) @ w2[e].double().T * w[t, j].double()[:, None])
    assert torch.equal(out, want.to(torch.bfloat16))


@pytest.mark.parametrize("T", [3, 60, 400])
def test_nan_stays_in_its_token(mxq, T):
    """E4M3 and scale NaN in a token's activations, and a NaN weight of a slot in use, reach that token's
    output alone."""
    E, H, I, k = 6, 256, 128, 2
    g = torch.Generator(device="cuda").manual_seed(T)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    mx = lambda t: mxq.MXFP8(*(lambda r: (r[0], r[1][2]))(mxq.quantize(t.contiguous(), layouts=(2,))))  # noqa: E731
    w13, w2 = mx(mxq.interleave_gate_up(rnd(E, I, H), rnd(E, I, H))), mx(rnd(E * H, I))
    q, sf = mxq.quantize(rnd(T, H), layouts=(0,))
    ids = torch.rand((T, E), generator=g, device="cuda").topk(k, dim=1).indices.to(torch.int32)
    w = torch.rand((T, k), generator=g, device="cuda")
    clean, out = (torch.empty((T, H), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    mxq.moe_experts_mxfp8(mxq.MXFP8(q, sf[0], 0), ids, w, w13, w2, clean)
    bad = sorted({0, T // 2, T - 1})
    q2, s2, w2nd = q.clone(), sf[0].clone().view(T, -1), w.clone()
    q2[0, 40] = 0x7F
    s2[T // 2, 3] = 0xFF
    w2nd[T - 1, 1] = float("nan")
    mxq.moe_experts_mxfp8(mxq.MXFP8(q2, s2.view(-1), 0), ids, w2nd, w13, w2, out)
    rest = [t for t in range(T) if t not in bad]
    assert torch.isfinite(clean.float()).all() and torch.equal(out[rest], clean[rest])
    assert torch.isnan(out[bad].float()).all()

"""moe_experts_mxfp8 on the GPU against the definition in 64 bits."""
import numpy as np
import pytest
import torch

from helpers import Guarded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mxq():
    from mxfp8_activation_quant_gb300 import build

    build.build()
    import mxfp8_activation_quant_gb300 as m

    assert torch.cuda.is_available(), "GPU tests need CUDA"
    m.load()
    return m


def values(q, sf):
    """E4M3 bytes and row-major UE8M0 bytes -> fp64."""
    scale = ((sf.long() + 896) << 52).view(torch.float64)
    return q.view(torch.float8_e4m3fn).double() * scale.view(q.shape[0], -1).repeat_interleave(32, dim=1)


class Model:
    def __init__(self, mxq, E, H, I, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.mxq, self.E, self.H, self.I, self.gen = mxq, E, H, I, g
        wg = torch.randn((E, I, H), generator=g, device="cuda").mul_(H ** -0.5).to(torch.bfloat16)
        wu = torch.randn((E, I, H), generator=g, device="cuda").mul_(H ** -0.5).to(torch.bfloat16)
        w2 = torch.randn((E * H, I), generator=g, device="cuda").mul_(I ** -0.5).to(torch.bfloat16)
        self.w13, self.w13v = self.mx(mxq.interleave_gate_up(wg, wu))
        self.w2, self.w2v = self.mx(w2)

    def mx(self, t, layout=2, ld=None):
        q, s = self.mxq.quantize(t, layouts=(0, 2))
        v = values(q, s[0])
        if ld is not None:
            wide = torch.zeros((q.shape[0], ld), dtype=torch.uint8, device="cuda")
            wide[:, :q.shape[1]] = q
            q = wide[:, :q.shape[1]]
        return self.mxq.MXFP8(q, s[layout], layout), v

    def x(self, T, layout=0, ld=None):
        return self.mx(torch.randn((T, self.H), generator=self.gen, device="cuda").to(torch.bfloat16), layout, ld)

    def route(self, T, k, spread=0.5):
        pop = torch.randn((T, self.E), generator=self.gen, device="cuda") + spread * torch.randn(
            self.E, generator=self.gen, device="cuda")
        top = pop.topk(min(k, self.E), dim=1)
        return top.indices.to(torch.int32).contiguous(), torch.softmax(top.values, 1).contiguous()

    def reference(self, xv, ids, w):
        out = torch.zeros((xv.shape[0], self.H), dtype=torch.float64, device="cuda")
        for e in range(self.E):
            t, j = torch.nonzero(ids == e, as_tuple=True)
            if not t.numel():
                continue
            gu = xv[t] @ self.w13v[e * 2 * self.I:(e + 1) * 2 * self.I].T
            g, u = gu[:, 0::2], gu[:, 1::2]
            h = (g * torch.sigmoid(g) * u).to(torch.bfloat16).contiguous()
            q, s = self.mxq.quantize(h, layouts=(0,))
            y = values(q, s[0]) @ self.w2v[e * self.H:(e + 1) * self.H].T
            out.index_add_(0, t, y * w[t, j].double()[:, None])
        return out

    def check(self, xm, xv, ids, w, **kw):
        T = xv.shape[0]
        out = Guarded(T * self.H * 2)
        status = self.mxq.new_status()
        o = out.view(torch.bfloat16, (T, self.H))
        self.mxq.moe_experts_mxfp8(xm, ids, w, self.w13, self.w2, o, status=status, **kw)
        self.mxq.check_status(status)
        assert out.intact()
        ref = self.reference(xv, ids, w)
        # Roundings: y to bf16 per expert and out to bf16, half a step (2^-9 at most, 2^-9 / sqrt 3 in
        # the mean) of a term each. An activation whose bf16 or E4M3 rounding falls the other way
        # (fp32 against fp64, about one in 10^4) moves by 2^-4 of itself: 2^-4 sqrt(10^-4) < 10^-3.
        norm = ref.norm()
        if norm > 0:
            assert ((o.double() - ref).norm() / norm).item() <= 4e-3
        # (one value: a group of 32 whose scale falls the other way at I = 128)
        rms = ref.square().mean(1, keepdim=True).sqrt()
        assert ((o.double() - ref).abs() <= 0.15 * rms + 2.0 ** -7 * ref.abs()).all()
        return o


@pytest.fixture(scope="module")
def small(mxq):
    return Model(mxq, E=12, H=512, I=256)


@pytest.mark.parametrize("layout", [0, 2])
@pytest.mark.parametrize("T,k", [(1, 1), (1, 8), (2, 3), (17, 2), (64, 4), (129, 3), (333, 5), (1000, 8), (2500, 12)])
def test_against_the_definition(small, T, k, layout):
    x, xv = small.x(T, layout)
    small.check(x, xv, *small.route(T, k))


@pytest.mark.parametrize("n", [1, 15, 16, 17, 31, 32, 33, 111, 112, 113, 127, 128, 129, 207, 208, 209, 223, 224, 225, 239, 416, 417, 448, 449])
def test_one_expert_with_n_tokens(small, n):
    """Token tiles at every border of the MMA's N, of the loads and of the scale atoms; the other
    experts are empty but for a last one with a single token."""
    ids = torch.full((n + 1, 1), 5, dtype=torch.int32, device="cuda")
    ids[-1] = 11
    x, xv = small.x(n + 1)
    small.check(x, xv, ids, torch.rand((n + 1, 1), generator=small.gen, device="cuda"))


@pytest.mark.parametrize("E,H,I", [(1, 128, 128), (3, 128, 640), (2, 640, 128), (40, 384, 128), (5, 2176, 384), (1, 1024, 2048)])
def test_widths(mxq, E, H, I):
    """Odd numbers of 128-row weight tiles, fewer k-blocks than stages, one expert."""
    m = Model(mxq, E, H, I, seed=E)
    for T, k in ((1, 1), (70, min(2, E)), (300, min(3, E))):
        x, xv = m.x(T)
        m.check(x, xv, *m.route(T, k))


def test_many_experts(mxq):
    m = Model(mxq, 1024, 128, 128, seed=9)
    x, xv = m.x(200)
    m.check(x, xv, *m.route(200, 8))


def test_slots_that_route_nowhere(small):
    x, xv = small.x(50)
    ids, w = small.route(50, 4)
    ids[3] = -1                 # a padding token
    ids[10:20, 2:] = -1
    ids[20, 1] = small.E        # not an expert either
    ids[21, 0] = 2 ** 31 - 1
    ids[22, 3] = -2 ** 31
    w[3] = float("nan")         # never read
    w[20, 1] = float("inf")
    o = small.check(x, xv, ids, torch.where((ids >= 0) & (ids < small.E), w, torch.zeros_like(w)))
    o2 = torch.empty_like(o)
    small.mxq.moe_experts_mxfp8(x, ids, w, small.w13, small.w2, o2)
    assert torch.equal(o, o2) and torch.all(o2[3] == 0)
    ids[:] = -1
    small.mxq.moe_experts_mxfp8(x, ids, w, small.w13, small.w2, o2)
    assert torch.all(o2 == 0)


def test_same_expert_twice_and_equal_rows(small):
    x, xv = small.x(30)
    ids = torch.full((30, 2), 4, dtype=torch.int32, device="cuda")
    w = torch.full((30, 2), 0.5, device="cuda")
    o = small.check(x, xv, ids, w)
    one = torch.empty_like(o)
    small.mxq.moe_experts_mxfp8(x, ids[:, :1].contiguous(), torch.ones((30, 1), device="cuda"), small.w13, small.w2, one)
    assert torch.equal(o, one)  # 0.5 y + 0.5 y = y exactly


def test_results_do_not_depend_on_the_batch(small):
    """A token's output is the same alone, in a batch, and in a batch in another order."""
    T, k = 260, 3
    x, xv = small.x(T)
    ids, w = small.route(T, k)
    o = small.check(x, xv, ids, w)
    perm = torch.randperm(T, generator=torch.Generator().manual_seed(1)).cuda()
    xp = small.mxq.MXFP8(x.data[perm].contiguous(), x.sf.view(T, -1)[perm].contiguous(), 0)
    op = torch.empty_like(o)
    small.mxq.moe_experts_mxfp8(xp, ids[perm].contiguous(), w[perm].contiguous(), small.w13, small.w2, op)
    assert torch.equal(op, o[perm])
    for t in (0, 101, 259):
        o1 = torch.empty((1, small.H), dtype=torch.bfloat16, device="cuda")
        x1 = small.mxq.MXFP8(x.data[t:t + 1], x.sf.view(T, -1)[t:t + 1].contiguous(), 0)
        small.mxq.moe_experts_mxfp8(x1, ids[t:t + 1], w[t:t + 1], small.w13, small.w2, o1)
        assert torch.equal(o1[0], o[t])


def test_strides_workspace_and_repeats(small):
    T, k = 77, 4
    x, xv = small.x(T, 2, ld=small.H + 48)
    ids, w = small.route(T, k)
    o = small.check(x, xv, ids, w)
    n = small.mxq.moe_workspace_bytes(T, k, small.E, small.H, small.I)
    ws = Guarded(n)  # filled with a canary: the contents need no clearing
    wide = torch.full((T, small.H + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    for _ in range(3):
        wide[:, :small.H] = float("nan")
        small.mxq.moe_experts_mxfp8(x, ids, w, small.w13, small.w2, wide[:, :small.H], workspace=ws.body)
        torch.cuda.synchronize()
        assert torch.equal(wide[:, :small.H], o) and torch.all(wide[:, small.H:] == 7.0)
    assert ws.intact()


def test_other_stream_and_graph(small):
    T, k = 40, 3
    x, xv = small.x(T)
    ids, w = small.route(T, k)
    o = small.check(x, xv, ids, w)
    s = torch.cuda.Stream()
    o2 = torch.zeros_like(o)
    torch.cuda.synchronize()
    small.mxq.moe_experts_mxfp8(x, ids, w, small.w13, small.w2, o2, stream=s)
    s.synchronize()
    assert torch.equal(o, o2)
    o2.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        small.mxq.moe_experts_mxfp8(x, ids, w, small.w13, small.w2, o2)
    ids.copy_(ids.flip(1))  # the graph reads the routing when it runs
    w.copy_(w.flip(1))
    want = small.check(x, xv, ids, w)
    for _ in range(3):
        o2.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(o2, want)


def test_two_streams_at_once(small):
    """Calls that overlap on two streams, each with a workspace of its own."""
    calls = []
    for T, k in ((700, 4), (33, 2)):
        x, xv = small.x(T)
        ids, w = small.route(T, k)
        want = small.check(x, xv, ids, w)
        ws = torch.empty(small.mxq.moe_workspace_bytes(T, k, small.E, small.H, small.I), dtype=torch.uint8, device="cuda")
        calls.append((x, ids, w, want, torch.zeros_like(want), ws, small.mxq.new_status(), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for x, ids, w, _, out, ws, status, stream in calls:
            small.mxq.moe_experts_mxfp8(x, ids, w, small.w13, small.w2, out, status=status, stream=stream, workspace=ws)
    torch.cuda.synchronize()
    for *_, want, out, ws, status, stream in calls:
        small.mxq.check_status(status)
        assert torch.equal(out, want)


def test_completes_while_other_work_holds_sms(small):
    """With most SMs held by another stream the call's blocks run in turns: no block waits for one that
    has not started, so it completes, with the same bytes."""
    import time

    T, k = 300, 4
    x, xv = small.x(T)
    ids, w = small.route(T, k)
    want = small.check(x, xv, ids, w)
    out, status = torch.zeros_like(want), small.mxq.new_status()
    ws = torch.empty(small.mxq.moe_workspace_bytes(T, k, small.E, small.H, small.I), dtype=torch.uint8, device="cuda")
    s_hold, s_call = torch.cuda.Stream(), torch.cuda.Stream()
    e_hold, e_call = torch.cuda.Event(), torch.cuda.Event()
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    torch.cuda.synchronize()
    small.mxq.selftest_hold_sms(sms // 2 - 12, 600_000, stream=s_hold)
    e_hold.record(s_hold)
    time.sleep(0.05)  # the holding kernel takes its SMs first
    small.mxq.moe_experts_mxfp8(x, ids, w, small.w13, small.w2, out, status=status, stream=s_call, workspace=ws)
    e_call.record(s_call)
    e_call.synchronize()
    held_still = not e_hold.query()
    torch.cuda.synchronize()
    small.mxq.check_status(status)
    assert held_still, "the call did not run beside the holding kernel"
    assert torch.equal(out, want)


def test_offsets_past_32_bits(mxq):
    """70000 tokens in 8 places: 2.3e9 elements of copied rows and of GEMM 2's output. A token's result
    does not depend on its batch, so a few tokens alone say what the large call has to give."""
    T, k, H = 70000, 8, 4096
    m = Model(mxq, 4, H, 128, seed=21)
    x, _ = m.mx(torch.randn((512, H), generator=m.gen, device="cuda").to(torch.bfloat16), 0)
    pick = torch.randint(0, 512, (T,), generator=m.gen, device="cuda")
    big = mxq.MXFP8(x.data[pick].contiguous(), x.sf.view(512, -1)[pick].contiguous(), 0)
    ids = torch.randint(0, 4, (T, k), generator=m.gen, device="cuda", dtype=torch.int32)
    w = torch.rand((T, k), generator=m.gen, device="cuda")
    out = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    status = mxq.new_status()
    mxq.moe_experts_mxfp8(big, ids, w, m.w13, m.w2, out, status=status)
    mxq.check_status(status)
    t = torch.cat([torch.arange(8), torch.randint(8, T - 8, (40,)), torch.arange(T - 8, T)]).cuda()
    few = torch.empty((t.numel(), H), dtype=torch.bfloat16, device="cuda")
    mxq.moe_experts_mxfp8(mxq.MXFP8(big.data[t].contiguous(), big.sf[t].contiguous(), 0), ids[t].contiguous(),
                          w[t].contiguous(), m.w13, m.w2, few)
    assert torch.equal(out[t], few)


def test_exact_integers(mxq):
    """Small whole numbers: every product and sum is exact, so silu's argument is chosen large (silu(g)
    = g to fp32 for g >= 32) and the result is the exact one, rounded to bf16."""
    E, H, I, T = 2, 256, 128, 150
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randint(0, 2, (T, H), generator=g, device="cuda").to(torch.bfloat16)
    x[:, 0] = 1.0
    wg = torch.zeros((E, I, H), dtype=torch.bfloat16, device="cuda")
    wg[:, :, 0] = 64.0
    wu = torch.zeros_like(wg)
    pick = torch.randint(1, H, (E, I), generator=g, device="cuda")
    wu.scatter_(2, pick[:, :, None], 1.0)
    w2 = torch.randint(-1, 2, (E * H, I), generator=g, device="cuda").to(torch.bfloat16)
    mx = lambda t: mxq.MXFP8(*(lambda r: (r[0], r[1][2]))(mxq.quantize(t.contiguous(), layouts=(2,))))  # noqa: E731
    ids = torch.randint(0, E, (T, 1), generator=g, device="cuda", dtype=torch.int32)
    out = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    mxq.moe_experts_mxfp8(mx(x), ids, torch.ones((T, 1), device="cuda"), mx(mxq.interleave_gate_up(wg, wu)), mx(w2), out)
    e = ids[:, 0].long()
    h = 64.0 * x.double().gather(1, pick[e])
    want = torch.bmm(w2.double().view(E, H, I)[e], h[:, :, None])[:, :, 0]
    assert torch.equal(out.double(), want.to(torch.bfloat16).double())

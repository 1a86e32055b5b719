"""The cache's operators together and with the output projection (examples/attention_half_layer.py): prompts written,
decode steps eager and captured, a prefix read back; each stage against its definition on the stage before it."""
import importlib.util
import os

import pytest
import torch

from kv_reference import attention, values

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    from mxfp8_activation_quant_gb300 import build

    build.build()
    assert torch.cuda.is_available(), "GPU tests need CUDA"
    spec = importlib.util.spec_from_file_location("attention_half_layer", os.path.join(ROOT, "examples", "attention_half_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


class Run:
    """Sequences with prompts of `lens` tokens in a layer's cache, and what the cache has to hold in rows of tokens."""

    def __init__(self, example, lens, width, seed):
        self.ex, self.lens, self.g = example, list(lens), torch.Generator(device="cuda").manual_seed(seed)
        B, page = len(lens), example.PAGE
        pages = B * width + 3
        self.layer = example.HalfLayer(example.Weights.random(), B, pages, width)
        self.layer.cache.data.fill_(0x7F)  # (NaN until written)
        self.layer.cache.sf.fill_(0xFF)
        self.layer.table.copy_(torch.randperm(pages, generator=self.g, device="cuda")[:B * width].view(B, width))
        self.rows = [self.normal(n, example.DIM) for n in lens]
        # the prompts as one batch, with rows that belong to nobody
        kv = torch.cat([*self.rows, self.normal(5, example.DIM)])
        slots = [self.slot(b, torch.arange(n, device="cuda")) for b, n in enumerate(lens)]
        self.layer.prefill(kv, torch.cat([*slots, torch.full((5,), -1, dtype=torch.int32, device="cuda")]).contiguous())
        self.q, self.kv = self.normal(B, example.HEADS, example.DIM), self.normal(B, example.DIM)
        self.slots = torch.empty(B, dtype=torch.int32, device="cuda")
        self.seq = torch.empty(B, dtype=torch.int32, device="cuda")

    def normal(self, *shape):
        return torch.randn(shape, generator=self.g, device="cuda").to(torch.bfloat16)

    def slot(self, b, pos):
        return (self.layer.table[b, pos // self.ex.PAGE] * self.ex.PAGE + pos % self.ex.PAGE).int()

    def advance(self):
        """The next step's inputs, in place."""
        self.q.copy_(self.normal(*self.q.shape))
        self.kv.copy_(self.normal(*self.kv.shape))
        for b, n in enumerate(self.lens):
            self.slots[b] = self.slot(b, torch.tensor([n], device="cuda"))[0]
            self.rows[b] = torch.cat([self.rows[b], self.kv[b:b + 1]])
            self.lens[b] = n + 1
        self.seq.copy_(torch.tensor(self.lens, dtype=torch.int32))

    def step(self):
        return self.layer.step(self.q, self.kv, self.slots, self.seq)

    def check(self):
        """The cache holds the tokens' quantized rows; o is within its tolerance of the attention over them, and
        its codes and the projection are those of a bf16 o from the same call."""
        m, layer, (B, H, D) = self.ex.mxq, self.layer, self.q.shape
        m.check_status(layer.status)
        for b, n in enumerate(self.lens):
            want, wsf = m.quantize(self.rows[b], layouts=(0,))
            at = self.slot(b, torch.arange(n, device="cuda")).long()
            assert torch.equal(layer.cache.data.view(-1, D)[at], want)
            assert torch.equal(layer.cache.sf.view(-1, D // 32)[at], wsf[0].view(n, -1))
        o = torch.empty_like(self.q)
        m.paged_attention_mxfp8(self.q, layer.cache, layer.table, self.seq, layer.scale, out=o)
        ref, _, tol, _ = attention(self.q, layer.cache.data, layer.cache.sf, None, None, layer.table, self.lens, layer.scale)
        assert bool(((o.double() - ref).abs() <= tol + 2.0 ** -8 * (ref.abs() + tol)).all())
        oq, osf = m.quantize(o.view(B, -1), layouts=(2,))
        assert torch.equal(layer.o, oq) and torch.equal(layer.osf, osf[2])
        out, s = torch.empty_like(layer.out), self.ex.synth
        m.o_proj_mxfp8(m.MXFP8(oq, osf[2]), layer.w.wa, layer.w.wb, B, s.G, s.NA, s.KA, s.NB, torch.empty_like(layer.z),
                       torch.empty_like(layer.zsf), out)
        assert torch.equal(layer.out, out)


@pytest.mark.parametrize("lens", [[1], [63, 64, 0, 200, 1], [(31 * i) % 150 for i in range(40)]])
def test_prompts_and_steps(example, lens):
    run = Run(example, lens, width=5, seed=len(lens))
    for _ in range(3):
        run.advance()
        run.step()
        run.check()


def test_captured_steps(example):
    """One graph, replayed as the sequences grow over a page's end; the same outputs as eager steps."""
    run, eager = (Run(example, [62, 127, 5, 300], width=6, seed=2) for _ in range(2))
    for r in (run, eager):
        r.advance()
        r.step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run.step()
    for _ in range(4):
        for r in (run, eager):
            r.advance()
        run.layer.out.zero_()
        graph.replay()
        want = eager.step()
        torch.cuda.synchronize()
        assert torch.equal(run.layer.out, want)
    run.check()


def test_prefix_read_back(example):
    """The start of a sequence, as the keys of a longer prompt's remaining tokens: the bf16 of what the cache holds."""
    m, run = example.mxq, Run(example, [100, 0, 70], width=2, seed=3)
    take, starts = [90, 0, 40], [0, 0, 30]
    out = torch.full((135, 1, example.DIM), 7.0, dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([0, 90, 90, 130], dtype=torch.int32, device="cuda")
    m.kv_read_bf16(run.layer.cache, run.layer.table, cu, out, starts=torch.tensor(starts, dtype=torch.int32, device="cuda"))
    at = 0
    for b, n in enumerate(take):
        if n:
            q, sf = m.quantize(run.rows[b][starts[b]:starts[b] + n].contiguous(), layouts=(0,))
            assert torch.equal(out[at:at + n, 0], values(q, sf[0].view(n, -1)).float().to(torch.bfloat16))
        at += n
    assert bool((out[130:] == 7.0).all())  # rows behind the last sequence stay


def test_example_runs(example, monkeypatch, capsys):
    monkeypatch.setattr("sys.argv", ["attention_half_layer.py", "--sequences", "3", "--tokens", "130"])
    example.main()
    assert "us per step" in capsys.readouterr().out

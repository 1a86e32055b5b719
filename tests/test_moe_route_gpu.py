"""moe_route on the GPU against the definition in 64 bits: ids exactly, weights within fp32."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

# score: exp within 2 ulp and three roundings (softmax: E additions and |l - m| 2^-24 more), the sum
# of k scores, a division and a product: below 2^-18 for E <= 1024 and |l| <= 16
RTOL = 2.0 ** -18


@pytest.fixture(scope="module")
def mxq():
    from mxfp8_activation_quant_gb300 import build

    build.build()
    import mxfp8_activation_quant_gb300 as m

    assert torch.cuda.is_available(), "GPU tests need CUDA"
    m.load()
    return m


def reference(logits, k, bias, scoring, groups, topk_groups, group_top, renormalize, scale):
    """The definition, row by row, in fp64 numpy."""
    l = logits.double().cpu().numpy()
    b = np.zeros(l.shape[1]) if bias is None else bias.double().cpu().numpy()
    T, E = l.shape
    ids, w = np.full((T, k), -1, np.int32), np.zeros((T, k))
    for t in range(T):
        there = l[t] > -np.inf
        if scoring == "sigmoid":
            with np.errstate(over="ignore"):
                s = 1.0 / (1.0 + np.exp(-l[t]))
        else:
            e = np.where(there, np.exp(l[t] - (l[t][there].max() if there.any() else 0.0)), 0.0)
            s = e / e.sum() if there.any() else e
        c = np.where(there, s + b, -np.inf)
        c = np.where(np.isnan(c), -np.inf, c)
        order = c if bias is not None else np.where(there, l[t], -np.inf)
        if groups > 1:
            g = np.sort(c.reshape(groups, -1), axis=1)[:, ::-1][:, :group_top]
            value = np.where(g[:, 0] == -np.inf, -np.inf, np.where(g > -np.inf, g, 0.0).sum(1))
            kept = [i for i in sorted(range(groups), key=lambda i: (-value[i], i))[:topk_groups] if value[i] > -np.inf]
            keep = np.zeros(groups, bool)
            keep[kept] = True
            order = np.where(np.repeat(keep, E // groups), order, -np.inf)
        top = [i for i in sorted(range(E), key=lambda i: (-order[i], i))[:k] if order[i] > -np.inf]
        ids[t, :len(top)] = top
        w[t, :len(top)] = s[top]
        if renormalize:
            w[t] /= w[t].sum() + 1e-20
    return ids, w * scale


def run(mxq, logits, k, **kw):
    T = logits.shape[0]
    ids = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), float("nan"), device="cuda")
    mxq.moe_route(logits, ids, w, **kw)
    torch.cuda.synchronize()
    return ids.cpu().numpy(), w.double().cpu().numpy()


def check(mxq, logits, k, **kw):
    full = dict(bias=None, scoring="sigmoid", groups=1, topk_groups=1, group_top=2, renormalize=True, scale=1.0)
    full.update(kw)
    ids, w = run(mxq, logits, k, **full)
    rid, rw = reference(logits, k, **full)
    assert np.array_equal(ids, rid), np.argwhere(ids != rid)[:4]
    np.testing.assert_allclose(w, rw, rtol=RTOL, atol=1e-30)


def gate(T, E, dtype=torch.float32, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    l = 1.5 * torch.randn((T, E), generator=g, device="cuda") + 0.5 * torch.randn(E, generator=g, device="cuda")
    return l.to(dtype), 0.1 * torch.randn(E, generator=g, device="cuda")


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T,E,k,groups,kept,top", [
    (1, 256, 8, 8, 4, 2), (1, 1, 1, 1, 1, 2), (5, 8, 2, 1, 1, 1), (33, 160, 6, 8, 3, 1), (130, 64, 8, 1, 1, 2),
    (67, 33, 5, 3, 2, 2), (9, 1024, 32, 32, 7, 2), (40, 512, 22, 4, 1, 2), (21, 384, 32, 1, 1, 2), (77, 96, 3, 32, 2, 2),
    (300, 256, 8, 8, 4, 2),
])
def test_against_the_definition(mxq, T, E, k, groups, kept, top, dtype, scoring):
    logits, bias = gate(T, E, dtype)
    for b in (None, bias):
        for renorm in (True, False):
            check(mxq, logits, k, bias=b, scoring=scoring, groups=groups, topk_groups=kept, group_top=top,
                  renormalize=renorm, scale=2.5)


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
def test_masked_logits_and_empty_rows(mxq, scoring):
    logits, bias = gate(64, 40, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    logits.masked_fill_(torch.rand(logits.shape, generator=g, device="cuda") < 0.85, float("-inf"))
    logits[7] = float("-inf")                        # nothing left
    logits[8, 1:] = float("-inf")                    # one expert left
    logits[9] = torch.finfo(torch.float32).min       # the type's lowest value is a value
    logits[10, ::2] = float("nan")
    for kw in (dict(), dict(groups=8, topk_groups=2, group_top=2), dict(groups=8, topk_groups=3, group_top=1)):
        for b in (None, bias):
            if scoring == "softmax" and b is not None:
                check(mxq, logits, 6, bias=b, scoring=scoring, renormalize=False, **kw)
            else:
                check(mxq, logits, 6, bias=b, scoring=scoring, **kw)


def test_masked_by_bias(mxq):
    logits, bias = gate(16, 24, seed=5)
    bias[3:20] = float("-inf")
    check(mxq, logits, 8, bias=bias)
    check(mxq, logits, 8, bias=bias, groups=4, topk_groups=2)


def test_ties_go_to_the_lowest_index(mxq):
    logits = torch.zeros((3, 128), device="cuda")
    logits[1, 100:] = 1.0
    logits[2, 5], logits[2, 90] = 2.0, 2.0
    zero = torch.zeros(128, device="cuda")
    for b in (None, zero):
        for kw in (dict(), dict(groups=8, topk_groups=2)):
            for scoring in ("sigmoid", "softmax"):
                check(mxq, logits, 4, bias=b, scoring=scoring, **kw)


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
def test_values_next_to_the_border(mxq, scoring):
    """Choices nearer than fp32 can tell: biases that bring an expert's score to within a few 2^-26
    of another's. The order is that of the exact values."""
    T, E = 256, 64
    logits, _ = gate(T, E, seed=6)
    logits[:] = logits[:1]  # one row's logits everywhere, so that the biases meet them
    l = logits[0].double().cpu()
    s = torch.sigmoid(l) if scoring == "sigmoid" else torch.softmax(l, 0)
    bias = (s.max() - s + 0.25).float().cuda()  # all choices equal up to the rounding of the bias
    check(mxq, logits, 8, bias=bias, scoring=scoring)
    check(mxq, logits, 8, bias=bias, scoring=scoring, groups=8, topk_groups=3)


@pytest.mark.parametrize("E,groups,kept,top", [(64, 8, 3, 2), (64, 8, 5, 1), (96, 8, 4, 2), (256, 8, 4, 2), (40, 5, 2, 2)])
@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
def test_groups_next_to_the_border(mxq, scoring, E, groups, kept, top):
    """Group values nearer than fp32 can tell: two experts of each group get biases that bring the sum
    of their choices to within a few 2^-26 of the other groups'; the rest stay far below."""
    T = 128
    logits, _ = gate(T, E, seed=E + kept)
    logits[:] = logits[:1]
    l = logits[0].double().cpu()
    s = torch.sigmoid(l) if scoring == "sigmoid" else torch.softmax(l, 0)
    g = torch.Generator().manual_seed(E)
    bias = torch.full((E,), -3.0, dtype=torch.float64)
    n = E // groups
    for i in range(groups):
        a, b = i * n + 1, i * n + n - 1
        d = 0.05 * torch.rand(1, generator=g).item() if top == 2 else 0.0
        bias[a], bias[b] = 1.0 + d - s[a], 1.0 - d - s[b]
    # logits of other rows differ in their last bits: the order of the exact sums changes with them
    logits += (torch.randint(-3, 4, (T, E), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
               * torch.finfo(torch.float32).eps)
    check(mxq, logits, 2 * kept, bias=bias.float().cuda(), scoring=scoring, groups=groups, topk_groups=kept, group_top=top)


def test_strided_rows_large_logits_and_stream(mxq):
    logits, bias = gate(50, 320, seed=7)
    view = (logits * 8.0)[:, 3:259]  # odd offset, row stride 320
    check(mxq, view, 8, bias=bias[3:259].contiguous(), groups=8, topk_groups=4)
    check(mxq, view.to(torch.bfloat16), 8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ids, w = torch.zeros((50, 8), dtype=torch.int32, device="cuda"), torch.zeros((50, 8), device="cuda")
    torch.cuda.synchronize()
    mxq.moe_route(view, ids, w, stream=s)
    s.synchronize()
    assert np.array_equal(ids.cpu().numpy(), reference(view, 8, None, "sigmoid", 1, 1, 2, True, 1.0)[0])


def test_infinite_logits(mxq):
    """+inf counts as the largest finite value: chosen first, and a softmax gives it everything."""
    logits, _ = gate(4, 32, seed=8)
    logits[:, 9] = float("inf")
    ids, w = run(mxq, logits, 2, scoring="softmax", renormalize=False)
    assert (ids[:, 0] == 9).all() and (w[:, 0] == 1.0).all() and (w[:, 1] == 0.0).all()
    ids, w = run(mxq, logits, 2, renormalize=False)
    assert (ids[:, 0] == 9).all() and (w[:, 0] == 1.0).all()

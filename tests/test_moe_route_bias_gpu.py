"""moe_route with biases that force or forbid experts: infinite ones and ones far from the scores."""
import numpy as np
import pytest
import torch

from test_moe_route_gpu import check, gate, mxq  # noqa: F401

pytestmark = pytest.mark.gpu
INF = float("inf")


@pytest.mark.parametrize("scoring", ["sigmoid", "softmax"])
@pytest.mark.parametrize("forced", [(0,), (9,), (0, 1), (3, 30), (0, 8, 16, 24), (5, 6, 7, 13, 14)])
@pytest.mark.parametrize("groups,kept,top", [(1, 1, 2), (4, 2, 1), (4, 2, 2), (4, 1, 2), (4, 3, 1)])
def test_forced_experts(mxq, groups, kept, top, forced, scoring):  # noqa: F811
    """A bias of +inf chooses its expert first (and its group), the lowest index among several."""
    logits, bias = gate(40, 32, seed=len(forced) + 10 * kept)
    bias[list(forced)] = INF
    check(mxq, logits, 6, bias=bias, scoring=scoring, groups=groups, topk_groups=kept, group_top=top)


@pytest.mark.parametrize("off", [-INF, -1e9, -3e38])
@pytest.mark.parametrize("E,groups,kept,top", [(256, 8, 4, 2), (256, 8, 3, 1), (96, 32, 5, 2), (160, 5, 2, 2), (256, 1, 1, 1)])
def test_experts_switched_off(mxq, E, groups, kept, top, off):  # noqa: F811
    logits, bias = gate(300, E, seed=E + kept)
    bias[torch.randperm(E, generator=torch.Generator().manual_seed(E))[:E // 8].cuda()] = off
    bias[:E // groups // 2] = off  # half of a group, or of all
    check(mxq, logits, 8, bias=bias, groups=groups, topk_groups=kept, group_top=top)


def test_all_far_below(mxq):  # noqa: F811
    """Choices whose sums lie outside fp32 are choices all the same."""
    logits, bias = gate(20, 64, seed=3)
    check(mxq, logits, 8, bias=torch.full_like(bias, -3e38), groups=8, topk_groups=2)
    check(mxq, logits, 8, bias=torch.full_like(bias, 3e38), groups=8, topk_groups=2)


@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_group_sums_past_fp32(mxq, sign):  # noqa: F811
    logits, bias = gate(20, 64, seed=4)
    for i in range(8):
        bias[8 * i + 2] = sign * (2.0e38 + 1e36 * ((5 * i) % 8))
        bias[8 * i + 3] = sign * 2.1e38
    if sign < 0:
        bias[bias > -1e30] = -3.3e38
    check(mxq, logits, 4, bias=bias, groups=8, topk_groups=2)
    check(mxq, logits, 4, bias=bias, groups=8, topk_groups=3, group_top=1)


@pytest.mark.parametrize("seed", range(6))
def test_biases_of_all_sizes(mxq, seed):  # noqa: F811
    """Magnitudes from 1e-8 to 1e30, both signs: a group's two largest may cancel."""
    rng = np.random.default_rng(seed)
    logits, _ = gate(100, 64, seed=seed)
    b = rng.choice([-1.0, 1.0], 64) * 10.0 ** rng.uniform(-8, 30 if seed % 2 else 4, 64)
    bias = torch.from_numpy(b.astype(np.float32)).cuda()
    for scoring in ("sigmoid", "softmax"):
        for kw in (dict(), dict(groups=8, topk_groups=3), dict(groups=32, topk_groups=5), dict(groups=8, topk_groups=3, group_top=1)):
            check(mxq, logits, 6, bias=bias, scoring=scoring, **kw)

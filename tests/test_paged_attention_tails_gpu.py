"""paged_attention_mxfp8 over many tokens of small probability beside one that leads: a long tail's part of the output."""
import math

import pytest
import torch

from test_paged_attention_gpu import mxq  # noqa: F401  (the module's fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv,G,D", [(1, 1, 128), (1, 16, 256), (1, 32, 512), (1, 64, 512)])
@pytest.mark.parametrize("below", [17.5, 22.5, 24.7, 25.5, 30.25])
def test_a_long_tail(mxq, below, kv, G, D):  # noqa: F811
    """A first token, of value 0, 2^below times as probable as each of the n - 1 others, of value 1: o is the others' share,
    w / (1 + w) with w = (n - 1) 2^-below. As many sequences as SMs, so that each is one CTA's from start to end.

    How far it may be off, of o:
    - an exponent: its score's fp32 roundings, 2^-22 of at most 31 (times ln 2), and the exponential's 2^-20
    - a probability in fp16, whose reference makes the largest one 2^7 at least: 2^-11 of it, and where it is not normal
      2^-25 of a unit of 2^-7, that is 2^-32 of the largest
    - the sums: the outputs take n / 16 additions, of 2^-23 of the sum so far each (an accumulator may cut off); the probabilities n / 128
      in a thread, of 2^-24 of the thread's sum so far. One thread's sum has the leader in it, that is nearly the whole sum: so 1 + w is off by
      n / 128 times 2^-24 of itself, not of w, and lse by as much
    - a rounding to bf16, 2^-8"""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    n, page = 1 << 17, 64
    kq = torch.zeros((2, page, kv, D), dtype=torch.uint8, device="cuda")
    vq = torch.full_like(kq, 0x38)                         # 1.0
    kq[0, 0], vq[0, 0] = 0x38, 0
    sf = torch.full((2, page, kv, D // 32), 127, dtype=torch.uint8, device="cuda")
    table = torch.ones((sms, n // page), dtype=torch.int32, device="cuda")
    table[:, 0] = 0
    seq = torch.full((sms,), n, dtype=torch.int32, device="cuda")
    q = torch.ones((sms, kv * G, D), dtype=torch.bfloat16, device="cuda")
    out, lse = torch.full_like(q, math.nan), torch.empty((sms, kv * G), device="cuda")
    scale = float(torch.tensor(below * math.log(2.0) / D, dtype=torch.float32))
    status = mxq.new_status()
    mxq.paged_attention_mxfp8(q, mxq.MXFP8Cache(kq, sf), table, seq, scale, v_cache=mxq.MXFP8Cache(vq, sf.clone()), out=out,
                              lse=lse, status=status)
    mxq.check_status(status)
    w = (n - 1) * math.exp(-scale * D)
    o = w / (1 + w)
    exponent = math.expm1(2.0 ** -22 * below) + 2.0 ** -20
    p = 2.0 ** below * 2.0 ** -32 + 2.0 ** -11
    sums = 2.0 ** -23 * (n / 16 + n / 128)
    tol = o * (exponent + p + sums)
    err = float((out.double() - o).abs().max())
    assert err <= tol + 2.0 ** -8 * (o + tol), f"{err / o} of the output, allowed {tol / o + 2.0 ** -8}"
    want = scale * D + math.log1p(w)
    assert float((lse.double() - want).abs().max()) <= o * exponent + 2.0 ** -24 * n / 128 + 2.0 ** -22 * want


@pytest.mark.parametrize("G,D", [(8, 128), (64, 512)])
def test_the_leader_comes_late(mxq, G, D):  # noqa: F811
    """The same sum with the leading token at the end, and scores that rise by less than the reference's slack on the way: a middle
    run of tokens 12 binary orders below the leader keeps the reference where the first run, 19 below, put it or moves it; either way the
    probabilities stay within fp16. Three runs of values 1, 2 and 4."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    page, runs = 64, [(300, 19.0, 1.0), (200, 12.0, 2.0), (1, 0.0, 4.0)]  # pages, binary orders below the leader, value
    # scores are 2^-j multiples of one key code: the leader's key 1.0, a run's key exact in E4M3 by its group's scale
    q = torch.ones((sms, G, D), dtype=torch.bfloat16, device="cuda")
    kq = torch.zeros((3, page, 1, D), dtype=torch.uint8, device="cuda")
    vq = torch.empty_like(kq)
    keys = [0.0, 7.0, 19.0]                                # in units of a binary order: 19 = leader, 19 - 12 = 7, 0
    for i, (key, (_, _, value)) in enumerate(zip(keys, runs)):
        first = torch.tensor(key, device="cuda") if key in (0.0, 7.0) else torch.tensor(18.0, device="cuda")
        rest = torch.tensor(1.0 if key == 19.0 else 0.0, device="cuda")
        kq[i, :, :, 0] = first.to(torch.float8_e4m3fn).view(torch.uint8)
        kq[i, :, :, 1] = rest.to(torch.float8_e4m3fn).view(torch.uint8)
        vq[i] = torch.tensor(value, device="cuda").to(torch.float8_e4m3fn).view(torch.uint8)
    sf = torch.full((3, page, 1, D // 32), 127, dtype=torch.uint8, device="cuda")
    table = torch.cat([torch.full((sms, n), i, dtype=torch.int32, device="cuda") for i, (n, _, _) in enumerate(runs)], dim=1)
    n = [300 * page, 200 * page, 1]
    seq = torch.full((sms,), sum(n), dtype=torch.int32, device="cuda")
    scale = float(torch.tensor(math.log(2.0), dtype=torch.float32))
    out = torch.full_like(q, math.nan)
    mxq.paged_attention_mxfp8(q, mxq.MXFP8Cache(kq, sf), table, seq, scale, v_cache=mxq.MXFP8Cache(vq, sf.clone()), out=out)
    weights = [c * math.exp(scale * (k - 19.0)) for c, k in zip(n, keys)]
    o = sum(w * v for w, (_, _, v) in zip(weights, runs)) / sum(weights)
    # (2^-19 and 2^-12 of the largest are normal numbers or off by 2^-32; the sums take n / 16 and n / 128 additions)
    rel = math.expm1(2.0 ** -22 * 19) + 2.0 ** -20 + 2.0 ** -11 + 2.0 ** -32 * 2.0 ** 19 + 2.0 ** -23 * (sum(n) / 16 + sum(n) / 128)
    tol = 2 * rel * o
    assert float((out.double() - o).abs().max()) <= tol + 2.0 ** -8 * (o + tol)

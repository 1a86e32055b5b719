"""include/mxq_moe.h: every declared symbol is exported and bad arguments are refused on the host
(these calls return before any CUDA work, so no GPU is needed)."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x7F0000000000  # never dereferenced: every call below fails validation first
OTHER = 0x7F1000000000


@pytest.fixture(scope="module")
def lib():
    from mxfp8_activation_quant_gb300 import build, moe

    build.build()
    return moe._fns()


def test_every_declared_symbol_is_exported(lib):
    from mxfp8_activation_quant_gb300 import moe

    text = open(os.path.join(ROOT, "include", "mxq_moe.h")).read()
    names = re.findall(r"MXQ_API\s+[\w\s\*]+?\b(\w+)\s*\(", text)
    assert set(names) == set(moe.SIGNATURES) and len(names) == 4
    for n in names:
        assert hasattr(lib, n), n


def norm_args(**kw):
    a = dict(x=FAKE, ldx=5120, res=OTHER, rt=0, ldr=5120, g=FAKE, eps=1e-6, T=4, H=5120, out=OTHER, ldro=5120, y=FAKE,
             yq=FAKE, pk=None, rm=FAKE, tl=None)
    a.update(kw)
    return (*a.values(), None)


@pytest.mark.parametrize("change,status", [
    (dict(x=None), 1), (dict(res=None), 1), (dict(g=None), 1), (dict(out=None), 1),
    (dict(rt=2), 1),                                     # unknown stream type
    (dict(y=None, yq=None, rm=None), 1),                 # no output
    (dict(rm=None), 1), (dict(yq=None), 1),              # y_q without scales, scales without y_q
    (dict(T=0), 1), (dict(T=-1), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
    (dict(H=5000, ldx=5120), 2), (dict(H=32768, ldx=32768, ldr=32768, ldro=32768), 2),
    (dict(ldx=5112), 2), (dict(ldr=5112), 2), (dict(ldro=5112), 2),
    (dict(H=96, pk=FAKE), 2),                            # packed scales, H % 128
    (dict(x=FAKE + 2), 3), (dict(res=OTHER + 8), 3), (dict(ldx=5124), 3), (dict(rt=1, ldr=5122), 3),
    (dict(ldro=5128), 1),                                # overlaps the residual without being it
    (dict(out=OTHER + 5120 * 2), 1),                     # the residual, one row on
    (dict(out=FAKE), 1),                                 # overwrites x
])
def test_add_rmsnorm_refusals(lib, change, status):
    assert lib.add_rmsnorm_dual_out(*norm_args(**change)) == status


def route_args(**kw):
    a = dict(l=FAKE, lt=1, ld=256, b=None, T=4, E=256, k=8, sc=0, g=8, tg=4, top=2, rn=1, s=1.0, ids=FAKE, w=FAKE)
    a.update(kw)
    return (*a.values(), None)


@pytest.mark.parametrize("change,status", [
    (dict(l=None), 1), (dict(ids=None), 1), (dict(w=None), 1), (dict(lt=7), 1), (dict(sc=2), 1),
    (dict(T=0), 1), (dict(E=0), 1), (dict(k=0), 1), (dict(g=0), 1), (dict(tg=0), 1), (dict(tg=9), 1),
    (dict(top=3), 1), (dict(s=float("inf")), 1), (dict(s=float("nan")), 1),
    (dict(E=1025, g=1, tg=1, ld=1025), 2), (dict(k=33), 2), (dict(E=250, ld=250), 2), (dict(ld=255), 2),
    (dict(E=64, g=32, tg=3, k=7, ld=64), 2),             # 3 groups of 2 hold 6 experts
    (dict(E=66, g=33, tg=4, ld=66), 2),                  # more than 32 groups
    (dict(l=FAKE + 2), 3), (dict(lt=0, l=FAKE + 1), 3), (dict(b=FAKE + 1), 3), (dict(ids=FAKE + 2), 3),
])
def test_route_refusals(lib, change, status):
    assert lib.moe_route(*route_args(**change)) == status


def test_experts_refusals(lib):
    from mxfp8_activation_quant_gb300._lib import MxTensorC

    def mx(rows, cols, layout=2, data=FAKE, sf=FAKE, ld=None):
        return MxTensorC(data, sf, layout, rows, cols, ld if ld is not None else cols)

    T, k, E, H, I = 4, 2, 8, 512, 256
    n = lib.mxq_moe_workspace_bytes(T, k, E, H, I)
    assert n > 0

    def call(x=mx(T, H, 0), ids=FAKE, w=FAKE, T=T, k=k, w13=mx(E * 2 * I, H), w2=mx(E * H, I), E=E, H=H, I=I, out=FAKE,
             ldo=H, ws=FAKE, wsn=n, st=None):
        B = ctypes.byref
        return lib.moe_experts_mxfp8(B(x) if x else None, ids, w, T, k, B(w13) if w13 else None, B(w2) if w2 else None, E,
                                     H, I, out, ldo, ws, wsn, st, None)

    assert call(x=None) == 1 and call(ids=None) == 1 and call(w=None) == 1 and call(out=None) == 1
    assert call(ws=None, wsn=0) == 1 and call(wsn=n - 1) == 1 and call(w13=None) == 1 and call(w2=None) == 1
    assert call(x=mx(T, H, 0, sf=None)) == 1
    assert call(T=0, x=mx(0, H, 0)) == 1 and call(k=0) == 1 and call(E=0) == 1
    assert call(x=mx(T, H, 1)) == 4 and call(w13=mx(E * 2 * I, H, 0)) == 4 and call(w2=mx(E * H, I, 1)) == 4
    assert call(k=65) == 2 and call(x=mx(T + 1, H, 0)) == 2 and call(w13=mx(E * I, H)) == 2
    assert call(w2=mx(E * H, I + 128)) == 2 and call(ldo=H - 8) == 2 and call(x=mx(T, H, 0, ld=H - 16)) == 2
    assert call(x=mx(T, 500, 0), H=500, w13=mx(E * 2 * I, 500), w2=mx(E * 500, I), ldo=504) == 2
    assert call(x=mx(T, H, 0, data=FAKE + 8)) == 3 and call(x=mx(T, H, 0, ld=H + 8)) == 3 and call(out=FAKE + 2) == 3
    assert call(ldo=H + 4) == 3 and call(ws=FAKE + 8) == 3 and call(ids=FAKE + 2) == 3 and call(w=FAKE + 1) == 3
    assert call(w13=mx(E * 2 * I, H, data=FAKE + 1)) == 3 and call(st=FAKE + 4) == 3


def test_workspace_of_invalid_shapes_is_zero(lib):
    w = lib.mxq_moe_workspace_bytes
    assert w(0, 2, 8, 512, 256) == 0 and w(4, 0, 8, 512, 256) == 0 and w(4, 65, 8, 512, 256) == 0
    assert w(4, 2, 1025, 512, 256) == 0 and w(4, 2, 8, 500, 256) == 0 and w(4, 2, 8, 512, 200) == 0
    assert w(1 << 24, 2, 8, 512, 256) == 0
    assert w(1, 1, 1, 128, 128) > 0 and w(1, 1, 1, 128, 128) % 16 == 0


def test_host_tensors_are_refused(lib):
    """The binding passes device pointers only: a host tensor is an error, not a CPU path."""
    import torch

    from mxfp8_activation_quant_gb300 import moe

    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensors"):
        moe.add_rmsnorm_dual_out(x, x.clone(), torch.ones(64, dtype=torch.bfloat16), 1e-6, x.clone(), x.clone())
    with pytest.raises(ValueError, match="device tensors"):
        moe.moe_route(torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2))
    q = moe.MXFP8(torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(16, dtype=torch.uint8), 0)
    w13 = moe.MXFP8(torch.zeros(256, 128, dtype=torch.uint8), torch.zeros(1024, dtype=torch.uint8))
    w2 = moe.MXFP8(torch.zeros(128, 128, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8))
    args = (torch.zeros(4, 1, dtype=torch.int32), torch.zeros(4, 1), w13, w2, torch.zeros(4, 128, dtype=torch.bfloat16))
    ws = torch.zeros(moe.moe_workspace_bytes(4, 1, 1, 128, 128), dtype=torch.uint8)
    with pytest.raises(ValueError, match="device tensors"):
        moe.moe_experts_mxfp8(q, *args, workspace=ws)
    with pytest.raises(AssertionError, match="scales"):
        moe.moe_experts_mxfp8(moe.MXFP8(q.data, q.sf[:8], 0), *args, workspace=ws)
    with pytest.raises(ValueError, match="sigmoid"):
        moe.moe_route(torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2), scoring="tanh")


def test_small_scale_buffers_are_refused(lib):
    import torch

    from mxfp8_activation_quant_gb300 import moe

    x = torch.zeros(5, 256, dtype=torch.bfloat16)
    q, g = torch.zeros(5, 256, dtype=torch.uint8), torch.ones(256, dtype=torch.bfloat16)
    for name, n in (("sf_rowmajor", 40), ("sf_packed", 64), ("sf_128x4", 1024)):
        with pytest.raises(AssertionError):
            moe.add_rmsnorm_dual_out(x, x.clone(), g, 1e-6, x.clone(), None, q, **{name: torch.zeros(n - 4, dtype=torch.uint8)})
        with pytest.raises(ValueError, match="device tensors"):
            moe.add_rmsnorm_dual_out(x, x.clone(), g, 1e-6, x.clone(), None, q, **{name: torch.zeros(n, dtype=torch.uint8)})


def test_interleave_gate_up():
    import torch

    from mxfp8_activation_quant_gb300 import interleave_gate_up

    g, u = torch.arange(2 * 3 * 4).view(2, 3, 4), -torch.arange(2 * 3 * 4).view(2, 3, 4)
    w = interleave_gate_up(g, u)
    assert w.shape == (12, 4) and torch.equal(w[0::2], g.reshape(6, 4)) and torch.equal(w[1::2], u.reshape(6, 4))

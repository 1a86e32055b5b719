"""ctypes binding of libmxq's mixture-of-experts operators (include/mxq_moe.h): argument
marshalling only, in the manner of ``_lib``.

The three calls make one half-layer of a mixture-of-experts decoder, activations MXFP8 between
them::

    add_rmsnorm_dual_out(x, h, gamma, eps, h, y, yq, sf_rowmajor=ysf)   # residual stream, norm
    moe_route(gate_logits, ids, weights, bias=balance)                  # k experts per token
    moe_experts_mxfp8(MXFP8(yq, ysf, SF_ROWMAJOR_U8), ids, weights, w13, w2, out)
"""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import _lib
from ._lib import I32, I64, MXFP8, P, SF_TILED_128X4, MxqError, _check, _ptr, _stream  # noqa: F401

TYPE_BF16, TYPE_FP32 = 0, 1
_TYPES = {torch.bfloat16: TYPE_BF16, torch.float32: TYPE_FP32}
_SCORING = {"sigmoid": 0, "softmax": 1}
_F32 = ctypes.c_float
_MXP = ctypes.POINTER(_lib.MxTensorC)

SIGNATURES = {
    "add_rmsnorm_dual_out": ([P, I64, P, I32, I64, P, _F32, I64, I64, P, I64, P, P, P, P, P, P], ctypes.c_int),
    "moe_route": ([P, I32, I64, P, I64, I32, I32, I32, I32, I32, I32, I32, _F32, P, P, P], ctypes.c_int),
    "mxq_moe_workspace_bytes": ([I64, I32, I32, I64, I64], I64),
    "moe_experts_mxfp8": ([_MXP, P, P, I64, I32, _MXP, _MXP, I32, I64, I64, P, I64, P, I64, P, P], ctypes.c_int),
}

_bound = None
# (looked up once; a torch without CUDA has neither, and no device tensor to call with)
_device, _raw_stream = getattr(torch._C, "_cuda_getDevice", None), getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _fns():
    """The loaded library with this module's signatures set."""
    global _bound
    lib = _lib._lib
    if lib is None or _bound is not lib:
        lib = _lib.load()
        for name, (args, res) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        _bound = lib
    return lib


def _host(*tensors):
    """For a call that was given a host tensor."""
    for t in tensors:
        _ptr(t)


# The first two calls take a few microseconds on the GPU for few tokens, less than their tensors take to
# be looked over here: so each property is asked for once, and pointers are taken in place.
def add_rmsnorm_dual_out(x: torch.Tensor, residual: torch.Tensor, gamma: torch.Tensor, eps: float,
                         residual_out: torch.Tensor, y: Optional[torch.Tensor] = None,
                         yq: Optional[torch.Tensor] = None, sf_packed=None, sf_rowmajor=None, sf_128x4=None,
                         stream=None) -> None:
    """residual_out = x + residual (bf16 or fp32 stream; may be `residual` itself), and its RMSNorm
    as bf16 y and/or MXFP8 yq with any subset of the three scale layouts."""
    shape = x.shape
    T, H = shape
    ldx, one = x.stride()
    ldr, one_r = residual.stride()
    ldo, one_o = residual_out.stride()
    st = residual.dtype
    assert x.dtype is torch.bfloat16 and st in _TYPES and residual_out.dtype is st and one == one_r == one_o == 1
    assert residual.shape == shape and residual_out.shape == shape
    assert gamma.dtype is torch.bfloat16 and gamma.numel() == H and gamma.is_contiguous()
    n = T * H
    assert y is None or (y.dtype is torch.bfloat16 and y.numel() == n and y.is_contiguous())
    assert yq is None or (yq.dtype is torch.uint8 and yq.numel() == n and yq.is_contiguous())
    assert sf_rowmajor is None or sf_rowmajor.nbytes * 32 >= n
    assert sf_packed is None or sf_packed.nbytes * 32 >= -(-T // 4) * 4 * H
    assert sf_128x4 is None or sf_128x4.nbytes >= -(-T // 128) * 128 * -(-H // 128) * 4
    if not (x.is_cuda and residual.is_cuda and gamma.is_cuda and residual_out.is_cuda):
        _host(x, residual, gamma, residual_out)
    status = _fns().add_rmsnorm_dual_out(
        x.data_ptr(), ldx, residual.data_ptr(), _TYPES[st], ldr, gamma.data_ptr(), eps, T, H, residual_out.data_ptr(), ldo,
        None if y is None else _ptr(y), None if yq is None else _ptr(yq), None if sf_packed is None else _ptr(sf_packed),
        None if sf_rowmajor is None else _ptr(sf_rowmajor), None if sf_128x4 is None else _ptr(sf_128x4),
        _raw_stream(_device()) if stream is None else _stream(stream))
    if status:
        _check(status, "add_rmsnorm_dual_out")


def moe_route(logits: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, bias: Optional[torch.Tensor] = None,
              scoring: str = "sigmoid", groups: int = 1, topk_groups: int = 1, group_top: int = 2,
              renormalize: bool = True, scale: float = 1.0, stream=None) -> None:
    """logits [T, E] (fp32 or bf16) -> ids int32 [T, k], weights fp32 [T, k]."""
    T, E = logits.shape
    ldl, one = logits.stride()
    rows, k = ids.shape
    assert logits.dtype in _TYPES and one == 1
    assert ids.dtype is torch.int32 and rows == T and ids.is_contiguous()
    assert weights.dtype is torch.float32 and weights.shape == ids.shape and weights.is_contiguous()
    assert bias is None or (bias.dtype is torch.float32 and bias.numel() == E and bias.is_contiguous())
    if scoring not in _SCORING:
        raise ValueError(f"scoring {scoring!r}: 'sigmoid' or 'softmax'")
    if not (logits.is_cuda and ids.is_cuda and weights.is_cuda):
        _host(logits, ids, weights)
    status = _fns().moe_route(
        logits.data_ptr(), _TYPES[logits.dtype], ldl, None if bias is None else _ptr(bias), T, E, k, _SCORING[scoring],
        groups, topk_groups, group_top, 1 if renormalize else 0, scale, ids.data_ptr(), weights.data_ptr(),
        _raw_stream(_device()) if stream is None else _stream(stream))
    if status:
        _check(status, "moe_route")


def moe_workspace_bytes(T: int, k: int, E: int, H: int, I: int) -> int:
    """Bytes of the workspace of moe_experts_mxfp8 on the current device; 0 for an invalid shape."""
    return int(_fns().mxq_moe_workspace_bytes(T, k, E, H, I))


def moe_experts_mxfp8(x: MXFP8, ids: torch.Tensor, weights: torch.Tensor, w13: MXFP8, w2: MXFP8, out: torch.Tensor,
                      status=None, stream=None, workspace: Optional[torch.Tensor] = None) -> None:
    """out[t] = sum_j weights[t, j] * W2_e(MXFP8(silu(g) * u)), (g, u) = W13_e x[t], e = ids[t, j].

    w13 [E * 2 I, H] (rows alternate gate, up: see interleave_gate_up), w2 [E * H, I]. workspace:
    None = allocated for this call on its stream, or a uint8 tensor of moe_workspace_bytes(...)."""
    lib = _fns()
    assert ids.dtype == torch.int32 and ids.dim() == 2 and ids.is_contiguous()
    assert weights.dtype == torch.float32 and weights.shape == ids.shape and weights.is_contiguous()
    T, k = ids.shape
    H, I = x.data.shape[1], w2.data.shape[1]
    E = w2.data.shape[0] // H if H else 0
    assert out.dtype == torch.bfloat16 and out.shape == (T, H) and out.stride(1) == 1
    n = lib.mxq_moe_workspace_bytes(T, k, E, H, I) if workspace is None else 0
    if workspace is None and n:
        if stream is None:
            workspace = torch.empty(n, dtype=torch.uint8, device=out.device)
        else:  # owned by the stream that uses it
            s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream))
            with torch.cuda.stream(s):
                workspace = torch.empty(n, dtype=torch.uint8, device=out.device)
    for m in (x, w13, w2):  # (weights' rows are multiples of 128)
        R, C = m.data.shape
        rows = R if m.layout == _lib.SF_ROWMAJOR_U8 else -(-R // 128) * 128
        assert m.sf.nbytes * 32 >= rows * C, "scales are missing"
        _host(m.data, m.sf)
    xc, ac, bc = x.c(), w13.c(), w2.c()
    _check(lib.moe_experts_mxfp8(ctypes.byref(xc), _ptr(ids), _ptr(weights), T, k, ctypes.byref(ac), ctypes.byref(bc),
                                 E, H, I, _ptr(out), out.stride(0), _ptr(workspace),
                                 0 if workspace is None else workspace.numel() * workspace.element_size(),
                                 _ptr(status), _stream(stream)), "moe_experts_mxfp8")


def interleave_gate_up(w_gate: torch.Tensor, w_up: torch.Tensor) -> torch.Tensor:
    """[E, I, H] gate and up projections -> [E * 2 I, H], rows alternating gate, up: the row order of
    moe_experts_mxfp8's w13 (quantize the result with F8_128x4 scales, once per model)."""
    E, I, H = w_gate.shape
    assert w_up.shape == w_gate.shape
    return torch.stack((w_gate, w_up), dim=2).reshape(E * 2 * I, H)

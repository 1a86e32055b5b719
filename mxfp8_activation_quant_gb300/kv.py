"""ctypes binding of libmxq's paged MXFP8 key-value cache (include/mxq_kv.h): argument marshalling only,
in the manner of ``_lib``.

The calls of a decode step around the attention; o leaves it as the operand of ``o_proj_mxfp8``::

    kv_write_mxfp8(k, slots, cache)                                # this step's tokens into their slots
    paged_attention_mxfp8(q, cache, block_table, seq_lens, scale, out_q=o, sf_128x4=osf)
    o_proj_mxfp8(MXFP8(o, osf), wa, wb, ...)
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import Optional

import torch

from . import _lib
from ._lib import I32, I64, P, _check, _ptr, _stream

_F32 = ctypes.c_float
_device = getattr(torch._C, "_cuda_getDevice", None)  # (a torch without CUDA has none, and no device tensor to call with)


class KvCacheC(ctypes.Structure):
    """The C struct mxq_kv_cache."""
    _fields_ = [("data", P), ("sf", P), ("pages", I64), ("page_size", I32), ("heads", I32), ("dim", I32),
                ("page_stride", I64), ("token_stride", I64), ("head_stride", I64),
                ("sf_page_stride", I64), ("sf_token_stride", I64), ("sf_head_stride", I64)]


_KVP = ctypes.POINTER(KvCacheC)

SIGNATURES = {
    "kv_write_mxfp8": ([P, I64, I64, _KVP, P, I64, I64, _KVP, P, I64, P], ctypes.c_int),
    "kv_read_bf16": ([_KVP, _KVP, P, I64, I32, P, P, I64, I64, P, P, P], ctypes.c_int),
    "mxq_paged_attention_workspace_bytes": ([I64, I32, I32, I32], I64),
    "paged_attention_mxfp8": ([P, I64, I64, _KVP, _KVP, P, I64, I32, P, I64, I32, _F32, P, P, P, P, P, P, P, I64, P, P],
                              ctypes.c_int),
}

_bound = None


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


def _here(t: torch.Tensor) -> None:
    """The calls launch on the current device, so that is where their tensors have to be."""
    _ptr(t)
    if t.get_device() != _device():
        raise ValueError("a tensor of another device than the current one")


@dataclass
class MXFP8Cache:
    """A paged cache: E4M3 bytes [pages, page_size, heads, dim] and UE8M0 scales [pages, page_size, heads,
    dim / 32] (uint8). Any strides with contiguous rows: a cache kept as [pages, heads, page_size, ..] is
    passed transposed(1, 2)."""
    data: torch.Tensor
    sf: torch.Tensor

    def c(self) -> KvCacheC:
        d, s = self.data, self.sf
        assert d.dtype is torch.uint8 and s.dtype is torch.uint8
        pages, page, heads, dim = d.shape
        ds, ss = d.stride(), s.stride()
        assert s.shape == (pages, page, heads, dim // 32) and ds[3] == 1 and (ss[3] == 1 or dim == 32)
        return KvCacheC(_ptr(d), _ptr(s), pages, page, heads, dim, ds[0], ds[1], ds[2], ss[0], ss[1], ss[2])

    @staticmethod
    def empty(pages: int, page_size: int, heads: int, dim: int, device="cuda") -> "MXFP8Cache":
        return MXFP8Cache(torch.empty((pages, page_size, heads, dim), dtype=torch.uint8, device=device),
                          torch.empty((pages, page_size, heads, dim // 32), dtype=torch.uint8, device=device))


def _rows(x: torch.Tensor, cache: MXFP8Cache, T: int):
    shape, st = x.shape, x.stride()
    assert x.dtype is torch.bfloat16 and shape[0] == T and shape[1:] == cache.data.shape[2:] and st[2] == 1
    return _ptr(x), st[0], st[1]


def _table(t: torch.Tensor, B: int):
    assert t.dtype is torch.int32 and t.dim() == 2 and t.shape[0] == B and (t.stride(1) == 1 or t.shape[1] == 1)
    return _ptr(t), t.stride(0), t.shape[1]


def kv_write_mxfp8(k: torch.Tensor, slots: torch.Tensor, k_cache: MXFP8Cache, v: Optional[torch.Tensor] = None,
                   v_cache: Optional[MXFP8Cache] = None, stream=None) -> None:
    """k bf16 [T, heads, dim] into the slots int32 [T] of the cache (-1: not written); v likewise."""
    T, = slots.shape
    assert slots.dtype is torch.int32 and slots.is_contiguous() and (v is None) == (v_cache is None)
    kp, kt, kh = _rows(k, k_cache, T)
    vp, vt, vh, vc = None, 0, 0, None
    if v is not None:
        vp, vt, vh = _rows(v, v_cache, T)
        vc = ctypes.byref(v_cache.c())
    _here(k)
    _check(_fns().kv_write_mxfp8(kp, kt, kh, ctypes.byref(k_cache.c()), vp, vt, vh, vc, _ptr(slots), T, _stream(stream)),
           "kv_write_mxfp8")


def kv_read_bf16(k_cache: MXFP8Cache, block_table: torch.Tensor, cu_rows: torch.Tensor, k_out: torch.Tensor,
                 v_cache: Optional[MXFP8Cache] = None, v_out: Optional[torch.Tensor] = None,
                 starts: Optional[torch.Tensor] = None, stream=None) -> None:
    """Rows cu_rows[b] .. cu_rows[b + 1] of k_out (and v_out), bf16 [rows, heads, dim], from the tokens of sequence
    b at starts[b] (0 without starts) and on; block_table int32 [B, width], cu_rows int32 [B + 1]."""
    B = cu_rows.shape[0] - 1
    assert cu_rows.dtype is torch.int32 and cu_rows.dim() == 1 and cu_rows.is_contiguous()
    assert starts is None or (starts.dtype is torch.int32 and starts.shape == (B,) and starts.is_contiguous())
    assert (v_out is None) == (v_cache is None)
    rows = k_out.shape[0]
    for x, c in ((k_out, k_cache),) + (() if v_out is None else ((v_out, v_cache),)):
        assert x.dtype is torch.bfloat16 and x.is_contiguous() and x.shape[0] == rows and x.shape[1:] == c.data.shape[2:]
    _here(k_out)
    _check(_fns().kv_read_bf16(ctypes.byref(k_cache.c()), None if v_cache is None else ctypes.byref(v_cache.c()),
                               *_table(block_table, B), _ptr(cu_rows), _ptr(starts), B, rows, _ptr(k_out), _ptr(v_out),
                               _stream(stream)), "kv_read_bf16")


def paged_attention_workspace_bytes(B: int, q_heads: int, kv_heads: int, dim: int) -> int:
    """Bytes of the workspace of paged_attention_mxfp8 on the current device; 0 for an invalid shape."""
    return int(_fns().mxq_paged_attention_workspace_bytes(B, q_heads, kv_heads, dim))


def paged_attention_mxfp8(q: torch.Tensor, k_cache: MXFP8Cache, block_table: torch.Tensor, seq_lens: torch.Tensor,
                          scale: float, v_cache: Optional[MXFP8Cache] = None, out: Optional[torch.Tensor] = None,
                          out_q: Optional[torch.Tensor] = None, sf_packed=None, sf_rowmajor=None, sf_128x4=None,
                          lse: Optional[torch.Tensor] = None, status=None, stream=None,
                          workspace: Optional[torch.Tensor] = None) -> None:
    """One new token's attention: q bf16 [B, q_heads, dim] over the first seq_lens[b] tokens of each sequence, as bf16
    out [B, q_heads, dim] and/or MXFP8 out_q [B, q_heads * dim] with any subset of the three scale layouts; lse
    fp32 [B, q_heads]. Without v_cache the values are the keys.

    workspace: None = allocated for this call on its stream, or a uint8 tensor of paged_attention_workspace_bytes(...)."""
    lib = _fns()
    B, H, D = q.shape
    qs = q.stride()
    kv = k_cache.data.shape[2]
    assert q.dtype is torch.bfloat16 and k_cache.data.shape[3] == D and qs[2] == 1
    assert seq_lens.dtype is torch.int32 and seq_lens.shape == (B,) and seq_lens.is_contiguous()
    n = B * H * D
    assert out is None or (out.dtype is torch.bfloat16 and out.numel() == n and out.is_contiguous())
    assert out_q is None or (out_q.dtype is torch.uint8 and out_q.numel() == n and out_q.is_contiguous())
    assert lse is None or (lse.dtype is torch.float32 and lse.numel() == B * H and lse.is_contiguous())
    assert sf_rowmajor is None or sf_rowmajor.nbytes * 32 >= n
    assert sf_packed is None or sf_packed.nbytes * 32 >= -(-B // 4) * 4 * H * D
    assert sf_128x4 is None or sf_128x4.nbytes * 32 >= -(-B // 128) * 128 * H * D
    _here(q)
    if workspace is None:
        size = lib.mxq_paged_attention_workspace_bytes(B, H, kv, D)
        if size:
            if stream is None:
                workspace = torch.empty(size, dtype=torch.uint8, device=q.device)
            else:  # owned by the stream that uses it
                s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream))
                with torch.cuda.stream(s):
                    workspace = torch.empty(size, dtype=torch.uint8, device=q.device)
    _check(lib.paged_attention_mxfp8(_ptr(q), qs[0], qs[1], ctypes.byref(k_cache.c()),
                                     None if v_cache is None else ctypes.byref(v_cache.c()), *_table(block_table, B),
                                     _ptr(seq_lens), B, H, scale, _ptr(out), _ptr(out_q), _ptr(sf_packed),
                                     _ptr(sf_rowmajor), _ptr(sf_128x4), _ptr(lse), _ptr(workspace),
                                     0 if workspace is None else workspace.nbytes, _ptr(status), _stream(stream)),
           "paged_attention_mxfp8")

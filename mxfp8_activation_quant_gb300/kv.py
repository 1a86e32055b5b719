"""ctypes binding of libmxq's paged MXFP8 key-value cache (include/mxq_kv.h): argument marshalling only,
in the manner of ``_lib``.

The calls of a decode step around the attention; o leaves it as the operand of ``o_proj_mxfp8``::

    kv_write_mxfp8(k, slots, cache)                                # this step's tokens into their slots
    paged_attention_mxfp8(q, cache, block_table, seq_lens, scale, out_q=o, sf_128x4=osf)
    o_proj_mxfp8(MXFP8(o, osf), wa, wb, ...)
"""
from __future__ import annotations

import ctypes
import struct
import threading
from dataclasses import dataclass
from typing import Optional

import torch

from . import _lib
from ._lib import I32, I64, P, _check, _ptr, _stream, torch_stream

_F32 = ctypes.c_float
_U8, _I32, _BF16, _FP32 = torch.uint8, torch.int32, torch.bfloat16, torch.float32
# (looked up once; a torch without CUDA has neither, and no device tensor to call with)
_device, _raw_stream = getattr(torch._C, "_cuda_getDevice", None), getattr(torch._C, "_cuda_getCurrentRawStream", None)
_capturing = torch.cuda.is_current_stream_capturing

# The C struct mxq_kv_cache as bytes: data, sf, pages, page_size, heads, dim, strides. (A few tokens take the GPU less
# than a ctypes structure takes to be filled.)
_CACHE = struct.Struct("@PPqiii4xqqqqqq")
_KVP = ctypes.c_char_p

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


def _refuse(*tensors: Optional[torch.Tensor]) -> None:
    """For a call whose tensors are not all on the current device, which is where it would launch."""
    for t in tensors:
        _ptr(t)
    raise ValueError("a tensor of another device than the current one")


def _on(dev: int, t: Optional[torch.Tensor]) -> Optional[int]:
    if t is None:
        return None
    if t.get_device() != dev:
        _refuse(t)
    return t.data_ptr()


@dataclass
class MXFP8Cache:
    """A paged cache: E4M3 bytes [pages, page_size, heads, dim] and UE8M0 scales [pages, page_size, heads,
    dim / 32] (uint8). Any strides with contiguous rows: a cache kept as [pages, heads, page_size, ..] is
    passed transposed(1, 2)."""
    data: torch.Tensor
    sf: torch.Tensor

    def c(self) -> bytes:
        d, s = self.data, self.sf
        pages, page, heads, dim = d.shape
        d0, d1, d2, one = d.stride()
        s0, s1, s2, one_s = s.stride()
        assert d.dtype is _U8 and s.dtype is _U8
        assert s.shape == (pages, page, heads, dim // 32) and one == 1 and (one_s == 1 or dim == 32)
        dev = d.get_device()
        if dev < 0 or s.get_device() != dev or dev != _device():
            _refuse(d, s)
        return _CACHE.pack(d.data_ptr(), s.data_ptr(), pages, page, heads, dim, d0, d1, d2, s0, s1, s2)

    @staticmethod
    def empty(pages: int, page_size: int, heads: int, dim: int, device="cuda") -> "MXFP8Cache":
        return MXFP8Cache(torch.empty((pages, page_size, heads, dim), dtype=torch.uint8, device=device),
                          torch.empty((pages, page_size, heads, dim // 32), dtype=torch.uint8, device=device))


def kv_write_mxfp8(k: torch.Tensor, slots: torch.Tensor, k_cache: MXFP8Cache, v: Optional[torch.Tensor] = None,
                   v_cache: Optional[MXFP8Cache] = None, stream=None) -> None:
    """k bf16 [T, heads, dim] into the slots int32 [T] of the cache (-1: not written); v likewise."""
    T, = slots.shape
    kt, kh, one = k.stride()
    assert slots.dtype is _I32 and slots.is_contiguous() and (v is None) == (v_cache is None)
    assert k.dtype is _BF16 and one == 1 and k.shape == (T, *k_cache.data.shape[2:])
    dev = k.get_device()
    if dev < 0 or slots.get_device() != dev or dev != _device():
        _refuse(k, slots)
    vp, vt, vh, vc = None, 0, 0, None
    if v is not None:
        vt, vh, one = v.stride()
        assert v.dtype is _BF16 and one == 1 and v.shape == (T, *v_cache.data.shape[2:])
        vp, vc = _on(dev, v), v_cache.c()
    status = _fns().kv_write_mxfp8(k.data_ptr(), kt, kh, k_cache.c(), vp, vt, vh, vc, slots.data_ptr(), T,
                                   _raw_stream(dev) if stream is None else _stream(stream))
    if status:
        _check(status, "kv_write_mxfp8")


def kv_read_bf16(k_cache: MXFP8Cache, block_table: torch.Tensor, cu_rows: torch.Tensor, k_out: torch.Tensor,
                 v_cache: Optional[MXFP8Cache] = None, v_out: Optional[torch.Tensor] = None,
                 starts: Optional[torch.Tensor] = None, stream=None) -> None:
    """Rows cu_rows[b] .. cu_rows[b + 1] of k_out (and v_out), bf16 [rows, heads, dim], from the tokens of sequence
    b at starts[b] (0 without starts) and on; block_table int32 [B, width], cu_rows int32 [B + 1]."""
    n, = cu_rows.shape
    B, rows = n - 1, k_out.shape[0]
    tb, width = block_table.shape
    ldt, one = block_table.stride()
    assert cu_rows.dtype is _I32 and cu_rows.is_contiguous()
    assert block_table.dtype is _I32 and tb == B and (one == 1 or width == 1)
    assert starts is None or (starts.dtype is _I32 and starts.shape == (B,) and starts.is_contiguous())
    assert (v_out is None) == (v_cache is None)
    assert k_out.dtype is _BF16 and k_out.is_contiguous() and k_out.shape == (rows, *k_cache.data.shape[2:])
    dev = k_out.get_device()
    if dev < 0 or block_table.get_device() != dev or cu_rows.get_device() != dev or dev != _device():
        _refuse(k_out, block_table, cu_rows)
    vp, vc = None, None
    if v_out is not None:
        assert v_out.dtype is _BF16 and v_out.is_contiguous() and v_out.shape == (rows, *v_cache.data.shape[2:])
        vp, vc = _on(dev, v_out), v_cache.c()
    status = _fns().kv_read_bf16(k_cache.c(), vc, block_table.data_ptr(), ldt, width, cu_rows.data_ptr(),
                                 _on(dev, starts), B, rows, k_out.data_ptr(), vp,
                                 _raw_stream(dev) if stream is None else _stream(stream))
    if status:
        _check(status, "kv_read_bf16")


_PER_THREAD = 2  # cudaStreamPerThread
_workspaces: dict = {}
_sharing = threading.Lock()  # held over a call with a kept workspace: two threads may call on one stream


def _workspace(dev: int, raw: int, size: int, stream):
    """(address, bytes) of the workspace kept for a stream, grown to `size` bytes where it is smaller; calls ordered on one
    stream may share it. Under capture a call gets one from the graph's own pool, so that no graph depends on what is kept here
    (freed on return: the pool gives it to work behind this call's only)."""
    if size <= 0:
        return None, 0
    if stream is not None:  # (memory is owned by the stream that uses it)
        with torch.cuda.stream(torch_stream(stream)):
            return _workspace(dev, raw, size, None)
    if _capturing():
        return torch.empty(size, dtype=_U8, device="cuda").data_ptr(), size
    if raw == _PER_THREAD:
        raise ValueError("the per-thread default stream is another one in each thread: give a workspace")
    ws = _workspaces.get((dev, raw))
    if ws is None or ws[1] < size:
        t = torch.empty(size, dtype=_U8, device="cuda")
        ws = _workspaces[dev, raw] = t.data_ptr(), size, t
    return ws[:2]


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

    workspace: None = one that this module keeps for the stream (allocated for this call under stream capture; the per-thread
    default stream has none), or a uint8 tensor of paged_attention_workspace_bytes(...)."""
    lib = _fns()
    B, H, D = q.shape
    ldq, ldqh, one = q.stride()
    tb, width = block_table.shape
    ldt, one_t = block_table.stride()
    shape = k_cache.data.shape
    assert q.dtype is _BF16 and shape[3] == D and one == 1
    assert seq_lens.dtype is _I32 and seq_lens.shape == (B,) and seq_lens.is_contiguous()
    assert block_table.dtype is _I32 and tb == B and (one_t == 1 or width == 1)
    n = B * H * D
    assert out is None or (out.dtype is _BF16 and out.numel() == n and out.is_contiguous())
    assert out_q is None or (out_q.dtype is _U8 and out_q.numel() == n and out_q.is_contiguous())
    assert lse is None or (lse.dtype is _FP32 and lse.numel() == B * H and lse.is_contiguous())
    assert sf_rowmajor is None or (sf_rowmajor.nbytes * 32 >= n and sf_rowmajor.is_contiguous())
    assert sf_packed is None or (sf_packed.nbytes * 32 >= -(-B // 4) * 4 * H * D and sf_packed.is_contiguous())
    assert sf_128x4 is None or (sf_128x4.nbytes * 32 >= -(-B // 128) * 128 * H * D and sf_128x4.is_contiguous())
    assert workspace is None or (workspace.dtype is _U8 and workspace.is_contiguous())
    assert status is None or (status.nbytes >= 4 and status.is_contiguous())
    dev = q.get_device()
    if dev < 0 or block_table.get_device() != dev or seq_lens.get_device() != dev or dev != _device():
        _refuse(q, block_table, seq_lens)
    kc, vc = k_cache.c(), None if v_cache is None else v_cache.c()
    outs = _on(dev, out), _on(dev, out_q), _on(dev, sf_packed), _on(dev, sf_rowmajor), _on(dev, sf_128x4), _on(dev, lse)
    args = (q.data_ptr(), ldq, ldqh, kc, vc, block_table.data_ptr(), ldt, width, seq_lens.data_ptr(), B, H, scale, *outs)
    status_at, raw = _on(dev, status), _raw_stream(dev) if stream is None else _stream(stream)
    if workspace is None:
        with _sharing:
            at, size = _workspace(dev, raw, lib.mxq_paged_attention_workspace_bytes(B, H, shape[2], D), stream)
            code = lib.paged_attention_mxfp8(*args, at, size, status_at, raw)
    else:
        code = lib.paged_attention_mxfp8(*args, _on(dev, workspace), workspace.nbytes, status_at, raw)
    if code:
        _check(code, "paged_attention_mxfp8")

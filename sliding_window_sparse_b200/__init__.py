"""Causal sliding-window attention for NVIDIA B200 (sm_100a).

A query at logical position i reads the keys at positions
max(0, i - W + 1) .. i (the window includes the query's own position), and
the softmax is taken over those pairs only.  Every step runs in the CUDA
kernels of ``libswa.so`` behind the C ABI of ``include/swa.h``; this module
only marshals torch tensors (device memory, current stream) into those calls.
The function names match the C entry points.  One addition sits above them:
``swa_attn_fwd_seq_parallel`` (module ``seq_parallel``) splits a sequence
along its length across ``torch.distributed`` ranks; it exchanges the W - 1
key/value rows before each shard and then calls ``swa_ring_write`` and
``swa_attn_chunk_ring``.

Layouts (row-major bf16): queries ``[B, H, rows, d]``, keys/values
``[B, Hkv, rows, d]``, ring caches ``[B, Hkv, W, d]``; query head h reads
key/value head ``h // (H // Hkv)``.  Paged caches are ``[n_pages, Hkv,
page_size, d]`` tensors of any strides (a token-major cache is passed as
``cache.transpose(1, 2)``) with an int32 page table ``[n_seq, max_pages]``.
"""

from __future__ import annotations

import ctypes
import functools
import math

import torch

from ._native import (Rotation, SwaError, check, lib, pack_paged_cache,  # noqa: F401
                      status_name)

__all__ = [
    "SwaError",
    "lib",
    "swa_block_meta",
    "swa_attn_fwd",
    "swa_attn_fwd_sink",
    "swa_attn_bwd",
    "swa_attn_varlen_bwd",
    "swa_attn_varlen",
    "swa_attn_chunk_ring",
    "swa_attn_chunk_ring_ragged",
    "swa_attn_chunk_ring_sink",
    "swa_attn_chunk_ring_split",
    "swa_chunk_split_workspace_bytes",
    "swa_ring_write",
    "swa_decode_workspace_bytes",
    "swa_attn_decode_ring",
    "swa_attn_decode_ring_sink",
    "swa_attn_decode_ring_static",
    "swa_ring_slot_positions",
    "swa_paged_append",
    "swa_chunk_paged_workspace_bytes",
    "swa_attn_chunk_paged",
    "swa_decode_paged_workspace_bytes",
    "swa_attn_decode_paged",
    "swa_selftest_wait",
    "swa_get_device_status",
    "swa_version",
    "swa_attn_fwd_seq_parallel",
]


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(device=None):
    return torch.cuda.current_stream(device).cuda_stream


def _need(t, name, dtype=torch.bfloat16, dims=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dims is not None and t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dims, got {t.dim()}")


def swa_version() -> int:
    return int(lib().swa_version())


def swa_block_meta(key_mode: int, n_q: int, n_k: int, W: int, tile_q: int, tile_k: int,
                   q_pos0: torch.Tensor | None = None, B: int | None = None,
                   classes: torch.Tensor | None = None, ranges: torch.Tensor | None = None,
                   device=None):
    """Tile classes (int8 [B,nqt,nkt]: 0 skip, 1 full, 2 partial) and ranges (int32 [B,nqt,4])."""
    if q_pos0 is not None:
        _need(q_pos0, "q_pos0", torch.int64, 1)
        B = q_pos0.numel()
        device = q_pos0.device
    if B is None:
        raise ValueError("B is required when q_pos0 is None")
    device = torch.device("cuda") if device is None else torch.device(device)
    nqt = (n_q + tile_q - 1) // tile_q
    nkt = ((n_k + tile_k - 1) // tile_k if key_mode == 0
           else (W + tile_k - 1) // tile_k + (n_q + tile_k - 1) // tile_k)
    if classes is None:
        classes = torch.empty((B, nqt, nkt), dtype=torch.int8, device=device)
    if ranges is None:
        ranges = torch.empty((B, nqt, 4), dtype=torch.int32, device=device)
    check("swa_block_meta", lib().swa_block_meta(key_mode, B, n_q, n_k, _ptr(q_pos0), W, tile_q,
                                                 tile_k, _ptr(classes), _ptr(ranges),
                                                 _stream(device)))
    return classes, ranges


def swa_attn_fwd(q, k, v, W: int, scale: float | None = None, out=None, lse=None,
                 return_lse: bool = False, n_sink: int = 0):
    """Prefill forward: q [B,H,N,d], k/v [B,Hkv,N,d] -> out [B,H,N,d] (and lse [B,H,N]).

    n_sink > 0 keeps keys 0..n_sink-1 visible to every later query (swa_attn_fwd_sink).
    """
    _need(q, "q", dims=4)
    _need(k, "k", dims=4)
    _need(v, "v", dims=4)
    B, H, N, d = q.shape
    Hkv = k.shape[1]
    if tuple(k.shape) != (B, Hkv, N, d) or tuple(v.shape) != (B, Hkv, N, d):
        raise ValueError("k and v must be [B, Hkv, N, d] matching q")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    _need(out, "out", dims=4)
    if return_lse and lse is None:
        lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device)
    if lse is not None:
        _need(lse, "lse", torch.float32, 3)
    if n_sink:
        check("swa_attn_fwd_sink",
              lib().swa_attn_fwd_sink(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), B, H, Hkv,
                                      N, d, W, n_sink, scale, _stream(q.device)))
    else:
        check("swa_attn_fwd", lib().swa_attn_fwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse),
                                                 B, H, Hkv, N, d, W, scale, _stream(q.device)))
    return (out, lse) if return_lse else out


def swa_attn_bwd(q, k, v, out, dout, lse, W: int, scale: float | None = None, dq=None, dk=None,
                 dv=None, workspace=None, n_sink: int = 0):
    """Gradients of swa_attn_fwd: returns (dq [B,H,N,d], dk, dv [B,Hkv,N,d]).

    out and lse are the forward's output and natural-log LSE; dout is the incoming gradient.
    n_sink > 0: gradients of swa_attn_fwd_sink with the same sinks (swa_attn_bwd_sink).
    """
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (out, "out"), (dout, "dout")):
        _need(t, n, dims=4)
    _need(lse, "lse", torch.float32, 3)
    B, H, N, d = q.shape
    Hkv = k.shape[1]
    if tuple(k.shape) != (B, Hkv, N, d) or tuple(v.shape) != (B, Hkv, N, d):
        raise ValueError("k and v must be [B, Hkv, N, d] matching q")
    if tuple(out.shape) != tuple(q.shape) or tuple(dout.shape) != tuple(q.shape):
        raise ValueError("out and dout must match q")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(v) if dv is None else dv
    need = int(lib().swa_attn_bwd_workspace_bytes(B, H, N))
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    if n_sink:
        check("swa_attn_bwd_sink",
              lib().swa_attn_bwd_sink(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(dout), _ptr(lse),
                                      _ptr(dq), _ptr(dk), _ptr(dv), B, H, Hkv, N, d, W, n_sink,
                                      scale, _ptr(workspace), ws_bytes, _stream(q.device)))
    else:
        check("swa_attn_bwd",
              lib().swa_attn_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(dout), _ptr(lse),
                                 _ptr(dq), _ptr(dk), _ptr(dv), B, H, Hkv, N, d, W, scale,
                                 _ptr(workspace), ws_bytes, _stream(q.device)))
    return dq, dk, dv


def swa_attn_varlen_bwd(q, k, v, cu_seqlens, max_seqlen: int, out, dout, lse, W: int,
                        scale: float | None = None, n_sink: int = 0, dq=None, dk=None, dv=None,
                        workspace=None):
    """Gradients of swa_attn_varlen: returns (dq [total,H,d], dk, dv [total,Hkv,d]).

    out and lse ([H, total]) are the forward's; dout is the incoming gradient.  Rows of
    tokens outside every sequence keep what dq / dk / dv held (zeros when allocated here).
    """
    for t, n in ((q, "q"), (k, "k"), (v, "v"), (out, "out"), (dout, "dout")):
        _need(t, n, dims=3)
    _need(cu_seqlens, "cu_seqlens", torch.int64, 1)
    _need(lse, "lse", torch.float32, 2)
    total, H, d = q.shape
    Hkv = k.shape[1]
    if tuple(k.shape) != (total, Hkv, d) or tuple(v.shape) != (total, Hkv, d):
        raise ValueError("k and v must be [total, Hkv, d] matching q")
    if tuple(out.shape) != tuple(q.shape) or tuple(dout.shape) != tuple(q.shape):
        raise ValueError("out and dout must match q")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dq = torch.zeros_like(q) if dq is None else dq
    dk = torch.zeros_like(k) if dk is None else dk
    dv = torch.zeros_like(v) if dv is None else dv
    need = int(lib().swa_attn_varlen_bwd_workspace_bytes(H, total))
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    check("swa_attn_varlen_bwd",
          lib().swa_attn_varlen_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens), _ptr(out),
                                    _ptr(dout), _ptr(lse), _ptr(dq), _ptr(dk), _ptr(dv),
                                    cu_seqlens.shape[0] - 1, total, max_seqlen, H, Hkv, d, W,
                                    n_sink, scale, _ptr(workspace),
                                    workspace.numel() * workspace.element_size(),
                                    _stream(q.device)))
    return dq, dk, dv


def swa_attn_varlen(q, k, v, cu_seqlens, max_seqlen: int, W: int, scale: float | None = None,
                    n_sink: int = 0, out=None, lse=None, return_lse: bool = False):
    """Packed prefill: q [total,H,d], k/v [total,Hkv,d], cu_seqlens int64 [n_seq+1] (device).

    Each sequence has its own positions and window; returns out [total,H,d] (and
    lse [H,total]).  Rows of tokens outside every sequence keep what `out` held.
    """
    _need(q, "q", dims=3)
    _need(k, "k", dims=3)
    _need(v, "v", dims=3)
    _need(cu_seqlens, "cu_seqlens", torch.int64, 1)
    total, H, d = q.shape
    Hkv = k.shape[1]
    if tuple(k.shape) != (total, Hkv, d) or tuple(v.shape) != (total, Hkv, d):
        raise ValueError("k and v must be [total, Hkv, d] matching q")
    n_seq = cu_seqlens.shape[0] - 1
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.zeros_like(q)
    _need(out, "out", dims=3)
    if return_lse and lse is None:
        lse = torch.zeros((H, total), dtype=torch.float32, device=q.device)
    if lse is not None:
        _need(lse, "lse", torch.float32, 2)
    check("swa_attn_varlen",
          lib().swa_attn_varlen(_ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens), _ptr(out), _ptr(lse),
                                n_seq, total, max_seqlen, H, Hkv, d, W, n_sink, scale,
                                _stream(q.device)))
    return (out, lse) if return_lse else out


def swa_attn_chunk_ring(q, k_new, v_new, k_ring, v_ring, q_start, scale: float | None = None,
                        update_ring: bool = False, out=None, lse=None, return_lse: bool = False,
                        k_sink=None, v_sink=None):
    """Chunked prefill on a ring cache: q [B,H,Tq,d], chunk k/v [B,Hkv,Tq,d], ring [B,Hkv,W,d].

    With k_sink / v_sink [B,Hkv,S,d] (positions 0..S-1) the sinks before each window
    are attended too (swa_attn_chunk_ring_sink).
    """
    for t, n in ((q, "q"), (k_new, "k_new"), (v_new, "v_new"), (k_ring, "k_ring"),
                 (v_ring, "v_ring")):
        _need(t, n, dims=4)
    _need(q_start, "q_start", torch.int64, 1)
    B, H, Tq, d = q.shape
    Hkv, W = k_ring.shape[1], k_ring.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if return_lse and lse is None:
        lse = torch.empty((B, H, Tq), dtype=torch.float32, device=q.device)
    if k_sink is not None:
        _need(k_sink, "k_sink", dims=4)
        _need(v_sink, "v_sink", dims=4)
        check("swa_attn_chunk_ring_sink",
              lib().swa_attn_chunk_ring_sink(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_ring),
                                             _ptr(v_ring), _ptr(k_sink), _ptr(v_sink),
                                             k_sink.shape[2], _ptr(q_start), _ptr(out), _ptr(lse),
                                             B, H, Hkv, Tq, d, W, scale, 1 if update_ring else 0,
                                             _stream(q.device)))
    else:
        check("swa_attn_chunk_ring",
              lib().swa_attn_chunk_ring(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_ring),
                                        _ptr(v_ring), _ptr(q_start), _ptr(out), _ptr(lse), B, H,
                                        Hkv, Tq, d, W, scale, 1 if update_ring else 0,
                                        _stream(q.device)))
    return (out, lse) if return_lse else out


def swa_attn_chunk_ring_ragged(q, k_new, v_new, k_ring, v_ring, q_start, chunk_len,
                               scale: float | None = None, update_ring: bool = False, out=None,
                               lse=None, return_lse: bool = False):
    """swa_attn_chunk_ring with chunk_len [B] valid rows per sequence (the rest is padding).

    Output rows at or beyond chunk_len[b] are left as they were in `out` (zeros when `out` is
    allocated here), likewise their lse entries.
    """
    for t, n in ((q, "q"), (k_new, "k_new"), (v_new, "v_new"), (k_ring, "k_ring"),
                 (v_ring, "v_ring")):
        _need(t, n, dims=4)
    _need(q_start, "q_start", torch.int64, 1)
    _need(chunk_len, "chunk_len", torch.int64, 1)
    B, H, Tq, d = q.shape
    Hkv, W = k_ring.shape[1], k_ring.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.zeros_like(q)
    if return_lse and lse is None:
        lse = torch.zeros((B, H, Tq), dtype=torch.float32, device=q.device)
    check("swa_attn_chunk_ring_ragged",
          lib().swa_attn_chunk_ring_ragged(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_ring),
                                           _ptr(v_ring), _ptr(q_start), _ptr(chunk_len),
                                           _ptr(out), _ptr(lse), B, H, Hkv, Tq, d, W, scale,
                                           1 if update_ring else 0, _stream(q.device)))
    return (out, lse) if return_lse else out


def swa_chunk_split_workspace_bytes(B: int, H: int, Hkv: int, Tq: int, d: int, W: int) -> int:
    return int(lib().swa_chunk_split_workspace_bytes(B, H, Hkv, Tq, d, W))


def swa_attn_chunk_ring_split(q, k_new, v_new, k_ring, v_ring, q_start, scale: float | None = None,
                              chunk_len=None, k_sink=None, v_sink=None, update_ring: bool = False,
                              out=None, lse=None, return_lse: bool = False, workspace=None):
    """Chunked prefill on a ring cache with a workspace that balances the work.

    The same results as swa_attn_chunk_ring / _ragged (chunk_len [B]) / _sink
    (k_sink, v_sink [B,Hkv,S,d]), within rounding: the last round of units is
    split across the SMs by key range and merged.  Rows past chunk_len[b] keep
    what `out` held (zeros when allocated here).
    """
    for t, n in ((q, "q"), (k_new, "k_new"), (v_new, "v_new"), (k_ring, "k_ring"),
                 (v_ring, "v_ring")):
        _need(t, n, dims=4)
    _need(q_start, "q_start", torch.int64, 1)
    if chunk_len is not None:
        _need(chunk_len, "chunk_len", torch.int64, 1)
    n_sink = 0
    if k_sink is not None:
        _need(k_sink, "k_sink", dims=4)
        _need(v_sink, "v_sink", dims=4)
        n_sink = k_sink.shape[2]
    B, H, Tq, d = q.shape
    Hkv, W = k_ring.shape[1], k_ring.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.zeros_like(q)
    if return_lse and lse is None:
        lse = torch.zeros((B, H, Tq), dtype=torch.float32, device=q.device)
    need = swa_chunk_split_workspace_bytes(B, H, Hkv, Tq, d, W)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    check("swa_attn_chunk_ring_split",
          lib().swa_attn_chunk_ring_split(_ptr(q), _ptr(k_new), _ptr(v_new), _ptr(k_ring),
                                          _ptr(v_ring), _ptr(k_sink), _ptr(v_sink), n_sink,
                                          _ptr(q_start), _ptr(chunk_len), _ptr(out), _ptr(lse), B,
                                          H, Hkv, Tq, d, W, scale, 1 if update_ring else 0,
                                          _ptr(workspace),
                                          workspace.numel() * workspace.element_size(),
                                          _stream(q.device)))
    return (out, lse) if return_lse else out


def swa_ring_write(k_new, v_new, k_ring, v_ring, q_start):
    """Write the chunk rows among the last W positions into slot position mod W (in place)."""
    for t, n in ((k_new, "k_new"), (v_new, "v_new"), (k_ring, "k_ring"), (v_ring, "v_ring")):
        _need(t, n, dims=4)
    _need(q_start, "q_start", torch.int64, 1)
    B, Hkv, T, d = k_new.shape
    W = k_ring.shape[2]
    check("swa_ring_write", lib().swa_ring_write(_ptr(k_new), _ptr(v_new), _ptr(k_ring),
                                                 _ptr(v_ring), _ptr(q_start), B, Hkv, T, d, W,
                                                 _stream(k_new.device)))


def swa_decode_workspace_bytes(B: int, H: int, Hkv: int, d: int, W: int) -> int:
    return int(lib().swa_decode_workspace_bytes(B, H, Hkv, d, W))


def swa_attn_decode_ring(q, k_ring, v_ring, pos, scale: float | None = None, workspace=None,
                         out=None, lse=None, return_lse: bool = False, k_sink=None,
                         v_sink=None):
    """Decode: q [B,H,d] at positions pos [B] over ring caches [B,Hkv,W,d] -> out [B,H,d].

    With k_sink / v_sink [B,Hkv,S,d] (positions 0..S-1) the sinks before the window are
    attended too (swa_attn_decode_ring_sink).
    """
    _need(q, "q", dims=3)
    _need(k_ring, "k_ring", dims=4)
    _need(v_ring, "v_ring", dims=4)
    _need(pos, "pos", torch.int64, 1)
    B, H, d = q.shape
    Hkv, W = k_ring.shape[1], k_ring.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    need = swa_decode_workspace_bytes(B, H, Hkv, d, W)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=q.device)
    if out is None:
        out = torch.empty_like(q)
    if return_lse and lse is None:
        lse = torch.empty((B, H), dtype=torch.float32, device=q.device)
    ws_bytes = workspace.numel() * workspace.element_size()
    if k_sink is not None:
        _need(k_sink, "k_sink", dims=4)
        _need(v_sink, "v_sink", dims=4)
        check("swa_attn_decode_ring_sink",
              lib().swa_attn_decode_ring_sink(_ptr(q), _ptr(k_ring), _ptr(v_ring), _ptr(k_sink),
                                              _ptr(v_sink), k_sink.shape[2], _ptr(pos), _ptr(out),
                                              _ptr(lse), B, H, Hkv, d, W, scale, _ptr(workspace),
                                              ws_bytes, _stream(q.device)))
    else:
        check("swa_attn_decode_ring",
              lib().swa_attn_decode_ring(_ptr(q), _ptr(k_ring), _ptr(v_ring), _ptr(pos),
                                         _ptr(out), _ptr(lse), B, H, Hkv, d, W, scale,
                                         _ptr(workspace), ws_bytes, _stream(q.device)))
    return (out, lse) if return_lse else out


def swa_attn_decode_ring_static(q, k_ring, v_ring, pos, scale: float | None = None, out=None,
                                lse=None, return_lse: bool = False):
    """Decode like swa_attn_decode_ring, for callers that cannot provide device scratch.

    The library keeps the split partials in its own fixed 16 MiB device array,
    so nothing is allocated for scratch; larger requests raise SwaError
    (SWA_ERR_WORKSPACE).
    Calls on one device share that array: do not let two of them overlap on
    the GPU (keep them on one stream or order them with events).  The first
    call on a device resolves the array's address; make it before any stream
    capture.
    """
    _need(q, "q", dims=3)
    _need(k_ring, "k_ring", dims=4)
    _need(v_ring, "v_ring", dims=4)
    _need(pos, "pos", torch.int64, 1)
    B, H, d = q.shape
    Hkv, W = k_ring.shape[1], k_ring.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is None:
        out = torch.empty_like(q)
    if return_lse and lse is None:
        lse = torch.empty((B, H), dtype=torch.float32, device=q.device)
    check("swa_attn_decode_ring_static",
          lib().swa_attn_decode_ring_static(_ptr(q), _ptr(k_ring), _ptr(v_ring), _ptr(pos),
                                            _ptr(out), _ptr(lse), B, H, Hkv, d, W, scale,
                                            _stream(q.device)))
    return (out, lse) if return_lse else out


def swa_ring_slot_positions(n_written, W: int, out=None):
    """int64 [B, W]: the logical position each ring slot holds after n_written[b] writes (-1 empty)."""
    _need(n_written, "n_written", torch.int64, 1)
    B = n_written.numel()
    if out is None:
        out = torch.empty((B, W), dtype=torch.int64, device=n_written.device)
    check("swa_ring_slot_positions", lib().swa_ring_slot_positions(
        B, _ptr(n_written), W, _ptr(out), _stream(n_written.device)))
    return out


# The paged calls serve single tokens, where the host's time counts: a check asks a tensor once
# and names it only when it fails, and the stream comes without a Python object around it.  (Torch
# keeps these two to itself, and a build without CUDA has neither: the public calls stand in.)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", _stream)
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_bf16 = torch.bfloat16
_INT_MAX = 0x7FFFFFFF


def _elsewhere(index, **named):
    """Raises for the first tensor that is not on CUDA device `index`."""
    for name, t in named.items():
        if t is not None and t.get_device() != index:
            raise ValueError(f"{name} must be on cuda:{index}, got {t.device}")


def _on(index, call, *args):
    """call(*args, stream) with CUDA device `index` current."""
    if _current_device() == index:
        return call(*args, _raw_stream(index))
    with torch.cuda.device(index):
        return call(*args, _raw_stream(index))


def _need_rows(t, name, shape):
    """bf16 [tokens, heads, d] whose token rows may lie apart (a slice of a fused projection)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda or t.dtype is not _bf16 or t.shape != shape:
        raise ValueError(f"{name} must be a bfloat16 CUDA tensor of shape {list(shape)}, got "
                         f"{t.dtype} {list(t.shape)} on {t.device}")
    total, heads, d = shape
    apart, head, one = t.stride()
    if one != 1 or (heads > 1 and head != d):
        raise ValueError(f"{name} must hold each token's [heads, d] contiguously")
    return apart if total > 1 else heads * d


def _need_list(t, name, dtype, length):
    """A contiguous CUDA vector of `length` entries."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda or t.dtype is not dtype or t.shape != (length,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor [{length}], got "
                         f"{t.dtype} {list(t.shape)} on {t.device}")


def _workspace_bytes(t):
    """Size of a caller's workspace, whose elements must not share memory (as expanded ones do)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("workspace must be a torch.Tensor")
    if not t.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return t.numel() * t.element_size()


def _need_like(t, name, dtype, shape):
    _need(t, name, dtype, len(shape))
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {list(shape)}, got {list(t.shape)}")


def _paged_cache(k_cache, v_cache, block_table, n_seq):
    """The cache's structure for the library, its heads and head dim."""
    if not (isinstance(k_cache, torch.Tensor) and isinstance(v_cache, torch.Tensor)
            and isinstance(block_table, torch.Tensor)):
        raise TypeError("k_cache, v_cache and block_table must be torch.Tensors")
    shape, strides = k_cache.shape, k_cache.stride()
    if not k_cache.is_cuda or k_cache.dtype is not _bf16 or v_cache.dtype is not _bf16 or \
            len(shape) != 4:
        raise ValueError("k_cache and v_cache must be bfloat16 CUDA tensors "
                         "[n_pages, Hkv, page_size, d]")
    n_pages, heads, page_size, d = shape
    page, head, slot, one = strides
    same = v_cache.shape == shape and v_cache.stride() == strides
    if n_pages == 1 or heads == 1 or page_size == 1:
        # the stride of a dimension of one entry says nothing: any valid one will do
        same = v_cache.shape == shape and all(n == 1 or a == b for n, a, b in
                                              zip(shape, strides, v_cache.stride()))
        page, head, slot = (d if n == 1 else s for n, s in zip(shape[:3], strides))
    if not same:
        raise ValueError("k_cache and v_cache must have the same shape and strides")
    if one != 1:
        raise ValueError("k_cache and v_cache must be contiguous in their last dimension")
    rows = block_table.shape
    if not block_table.is_cuda or block_table.dtype is not torch.int32 or len(rows) != 2 or \
            rows[0] != n_seq:
        raise ValueError(f"block_table must be an int32 CUDA tensor [{n_seq}, max_pages]")
    max_pages = rows[1]
    apart, one = block_table.stride()
    if one != 1 and max_pages > 1:
        raise ValueError("block_table must be contiguous along a row")
    return (pack_paged_cache(k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(), page,
                             head, slot, n_pages, max_pages, apart if n_seq > 1 else max_pages,
                             min(page_size, _INT_MAX)), heads, d)


def swa_paged_append(k_new, v_new, k_cache, v_cache, block_table, cu_seqlens, q_start, q=None,
                     q_out=None, inv_freq=None, interleaved: bool = False, positions=None,
                     pair_axis=None):
    """Append packed new tokens to a paged cache, rotating keys (and queries) on the way.

    k_new, v_new [total, Hkv, d] (rows may lie apart, as in a slice of a fused projection) go to
    the pages of their sequences: token t of sequence b (cu_seqlens int64 [n_seq + 1]) to position
    q_start[b] + t - cu_seqlens[b], page block_table[b, position // page_size].  inv_freq float32
    [rot_dim / 2] turns the first rot_dim elements of every key and query head by position *
    inv_freq[i], in pairs (i, i + rot_dim / 2) or, when interleaved, (2i, 2i + 1); positions
    int64 [total] or [n_axes, total] and pair_axis int32 [rot_dim / 2] give each pair a position
    of its own (time, height, width).  Returns the rotated queries: q_out, a new tensor when None
    (zeros where a token writes no slot), or None when q is None.  q_out may be q itself.
    """
    if not isinstance(k_new, torch.Tensor) or k_new.dim() != 3:
        raise ValueError("k_new must be [total, Hkv, d]")
    total, Hkv, d = shape = k_new.shape
    ks = _need_rows(k_new, "k_new", shape)
    vs = _need_rows(v_new, "v_new", shape)
    n_seq = q_start.shape[0] if isinstance(q_start, torch.Tensor) and q_start.dim() == 1 else 0
    _need_list(q_start, "q_start", torch.int64, n_seq)
    _need_list(cu_seqlens, "cu_seqlens", torch.int64, n_seq + 1)
    cache, heads, dk = _paged_cache(k_cache, v_cache, block_table, n_seq)
    if heads != Hkv or dk != d:
        raise ValueError(f"the cache has {heads} heads of {dk}, expected {Hkv} of {d}")
    H, qs, qos, zero_rest = 0, 0, 0, False
    if q is not None:
        if not isinstance(q, torch.Tensor) or q.dim() != 3:
            raise ValueError("q must be [total, H, d]")
        H = q.shape[1]
        qs = _need_rows(q, "q", (total, H, d))
        if q_out is None:
            zero_rest = True
            q_out = q.new_empty((total, H, d))
            qos = H * d
        else:
            qos = _need_rows(q_out, "q_out", (total, H, d))
    elif q_out is not None:
        raise ValueError("q_out without q")
    rotation = None
    if inv_freq is not None:
        _need(inv_freq, "inv_freq", torch.float32, 1)
        half = inv_freq.shape[0]
        n_axes = 0
        if positions is not None:
            _need(positions, "positions", torch.int64)
            if positions.dim() not in (1, 2) or positions.shape[-1] != total:
                raise ValueError(f"positions must be [{total}] or [n_axes, {total}]")
            n_axes = positions.shape[0] if positions.dim() == 2 else 1
        if pair_axis is not None:
            if positions is None:
                raise ValueError("pair_axis without positions")
            _need_list(pair_axis, "pair_axis", torch.int32, half)
        rotation = Rotation(_ptr(inv_freq), _ptr(positions), _ptr(pair_axis), total, 2 * half,
                            1 if interleaved else 0, n_axes)
    elif positions is not None or pair_axis is not None:
        raise ValueError("positions and pair_axis need inv_freq")
    index = k_new.get_device()
    if not (v_new.get_device() == k_cache.get_device() == v_cache.get_device()
            == block_table.get_device() == cu_seqlens.get_device() == q_start.get_device()
            == index and (q is None or q.get_device() == q_out.get_device() == index)
            and (rotation is None or inv_freq.get_device() == index)
            and (positions is None or positions.get_device() == index)
            and (pair_axis is None or pair_axis.get_device() == index)):
        _elsewhere(index, v_new=v_new, k_cache=k_cache, v_cache=v_cache, block_table=block_table,
                   cu_seqlens=cu_seqlens, q_start=q_start, q=q, q_out=q_out, inv_freq=inv_freq,
                   positions=positions, pair_axis=pair_axis)
    check("swa_paged_append",
          _on(index, lib().swa_paged_append, k_new.data_ptr(), ks, v_new.data_ptr(), vs, _ptr(q),
              qs, _ptr(q_out), qos, cache,
              ctypes.byref(rotation) if rotation else None, cu_seqlens.data_ptr(),
              q_start.data_ptr(), n_seq, total, H, Hkv, d, 1 if zero_rest else 0))
    return q_out


@functools.lru_cache(maxsize=256)
def swa_chunk_paged_workspace_bytes(n_seq: int, total: int, H: int, Hkv: int, d: int) -> int:
    return int(lib().swa_chunk_paged_workspace_bytes(n_seq, total, H, Hkv, d))


def swa_attn_chunk_paged(q, k_cache, v_cache, block_table, cu_seqlens, q_start, W: int,
                         scale: float | None = None, n_sink: int = 0, out=None, lse=None,
                         return_lse: bool = False, workspace=None):
    """Attention of packed new tokens q [total, H, d] over a paged cache -> out [total, H, d].

    Query t of sequence b (cu_seqlens int64 [n_seq + 1]) sits at p = q_start[b] + t and reads the
    cached keys j <= p of its own sequence with j >= p - W + 1 or j < n_sink (its own key and
    those of the chunk are in the cache already, see swa_paged_append).  lse is [H, total].  Rows
    of tokens outside every sequence, or of a sequence that is skipped because its offsets or
    start are out of range, keep what out and lse held (zeros when allocated here).
    """
    _need(q, "q", dims=3)
    total, H, d = q.shape
    n_seq = q_start.shape[0] if isinstance(q_start, torch.Tensor) and q_start.dim() == 1 else 0
    _need_list(q_start, "q_start", torch.int64, n_seq)
    _need_list(cu_seqlens, "cu_seqlens", torch.int64, n_seq + 1)
    cache, Hkv, dk = _paged_cache(k_cache, v_cache, block_table, n_seq)
    if dk != d:
        raise ValueError(f"the cache has heads of {dk}, q of {d}")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    new_out, new_lse = out is None, return_lse and lse is None
    if not new_out:
        _need(out, "out", dims=3)
        if out.shape != q.shape:
            raise ValueError("out must match q")
    if lse is not None:
        _need_like(lse, "lse", torch.float32, (H, total))
    index = q.get_device()
    if not (k_cache.get_device() == v_cache.get_device() == block_table.get_device()
            == cu_seqlens.get_device() == q_start.get_device() == index):
        _elsewhere(index, k_cache=k_cache, v_cache=v_cache, block_table=block_table,
                   cu_seqlens=cu_seqlens, q_start=q_start)
    if workspace is not None:
        ws_bytes = _workspace_bytes(workspace)
    if not (new_out and lse is None and workspace is None):
        _elsewhere(index, out=out, lse=lse, workspace=workspace)
    # what is allocated here is zeroed by the call where no sequence writes, unless the other of
    # the two is the caller's: then its rows stay, and ours are zeroed first
    zero_rest = new_out and (new_lse or lse is None)
    if new_out:
        out = torch.empty_like(q) if zero_rest else torch.zeros_like(q)
    if new_lse:
        lse = q.new_empty((H, total), dtype=torch.float32)
        if not zero_rest:
            lse.zero_()
    if workspace is None:
        ws_bytes = max(swa_chunk_paged_workspace_bytes(n_seq, total, H, Hkv, d), 256)
        workspace = q.new_empty(ws_bytes, dtype=torch.uint8)
    check("swa_attn_chunk_paged",
          _on(index, lib().swa_attn_chunk_paged, q.data_ptr(), cache,
              cu_seqlens.data_ptr(), q_start.data_ptr(), out.data_ptr(), _ptr(lse), n_seq, total,
              H, Hkv, d, W, n_sink, scale, 1 if zero_rest else 0, workspace.data_ptr(),
              ws_bytes))
    return (out, lse) if return_lse else out


@functools.lru_cache(maxsize=256)
def swa_decode_paged_workspace_bytes(B: int, H: int, Hkv: int, d: int) -> int:
    return int(lib().swa_decode_paged_workspace_bytes(B, H, Hkv, d))


def swa_attn_decode_paged(q, k_cache, v_cache, block_table, pos, W: int,
                          scale: float | None = None, n_sink: int = 0, workspace=None, out=None,
                          lse=None, return_lse: bool = False):
    """Decode over a paged cache: q [B, H, d] at positions pos [B] -> out [B, H, d], lse [B, H].

    The query of sequence b reads the cached keys j <= pos[b] with j >= pos[b] - W + 1 or
    j < n_sink.  pos[b] = -1 marks a padded row: output zero, lse -infinity.
    """
    _need(q, "q", dims=3)
    B, H, d = q.shape
    _need_list(pos, "pos", torch.int64, B)
    cache, Hkv, dk = _paged_cache(k_cache, v_cache, block_table, B)
    if dk != d:
        raise ValueError(f"the cache has heads of {dk}, q of {d}")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    if out is not None:
        _need(out, "out", dims=3)
        if out.shape != q.shape:
            raise ValueError("out must match q")
    if lse is not None:
        _need_like(lse, "lse", torch.float32, (B, H))
    index = q.get_device()
    if not (k_cache.get_device() == v_cache.get_device() == block_table.get_device()
            == pos.get_device() == index):
        _elsewhere(index, k_cache=k_cache, v_cache=v_cache, block_table=block_table, pos=pos)
    if workspace is not None:
        ws_bytes = _workspace_bytes(workspace)
    if not (out is None and lse is None and workspace is None):
        _elsewhere(index, out=out, lse=lse, workspace=workspace)
    if out is None:
        out = torch.empty_like(q)
    if return_lse and lse is None:
        lse = q.new_empty((B, H), dtype=torch.float32)
    if workspace is None:
        ws_bytes = max(swa_decode_paged_workspace_bytes(B, H, Hkv, d), 256)
        workspace = q.new_empty(ws_bytes, dtype=torch.uint8)
    check("swa_attn_decode_paged",
          _on(index, lib().swa_attn_decode_paged, q.data_ptr(), cache,
              pos.data_ptr(), out.data_ptr(), _ptr(lse), B, H, Hkv, d, W, n_sink, scale,
              workspace.data_ptr(), ws_bytes))
    return (out, lse) if return_lse else out


def swa_selftest_wait(limit_ns: int, arrive: bool = False, device=None):
    """Run the library's bounded device wait in a one-CTA kernel of its own.

    arrive=False: nobody arrives on the barrier, so the wait gives up after
    limit_ns and swa_get_device_status() then reports SWA_ERR_TIMEOUT (5).
    Returns int32 [5] on the device: lanes of warps 0..3 whose wait succeeded,
    then the elapsed microseconds.
    """
    device = torch.device("cuda") if device is None else torch.device(device)
    res = torch.zeros(5, dtype=torch.int32, device=device)
    check("swa_selftest_wait", lib().swa_selftest_wait(int(limit_ns), 1 if arrive else 0,
                                                       _ptr(res), _stream(device)))
    return res


def swa_get_device_status(stream=None) -> int:
    """Synchronise the stream and return (and clear) the device status word as a status code."""
    s = _stream() if stream is None else stream
    return int(lib().swa_get_device_status(s))


def swa_attn_fwd_seq_parallel(q, k, v, W: int, scale: float | None = None, out=None,
                              return_lse: bool = False, group=None, ring_k=None, ring_v=None):
    """Prefill of a sequence split along its length across ranks (see ``seq_parallel``)."""
    from .seq_parallel import swa_attn_fwd_seq_parallel as run

    return run(q, k, v, W, scale=scale, out=out, return_lse=return_lse, group=group,
               ring_k=ring_k, ring_v=ring_v)

"""ctypes binding of the attention calls: ordinary and differential softmax
attention over whole sequences, its gradients, the decode step over a paged
cache, and the cache's filling.

As in _block, this is argument marshalling only, and sequence tensors and caches
may have any strides as long as the elements of a row are contiguous.
"""
from __future__ import annotations

from typing import Optional, Tuple, Union

import torch

from ._block import _call, _dtype, _out, _p, _pack, _rows, _workspace
from ._lib import _sizes, load


def _i32(t: Optional[torch.Tensor], shape, like: torch.Tensor, name: str) -> Optional[torch.Tensor]:
    """Lengths, positions or page numbers: contiguous int32 on the same device."""
    if t is not None and (t.dtype != torch.int32 or t.shape != shape or t.get_device() != like.get_device() or
                          not t.is_contiguous()):
        raise ValueError(f"{name} must be contiguous int32 {tuple(shape)} on {like.device}")
    return t


def _weights(t: Optional[torch.Tensor], H: int, like: torch.Tensor, name: str) -> Optional[torch.Tensor]:
    if t is not None and (t.dtype != torch.float32 or t.shape != (H,) or t.get_device() != like.get_device() or
                          not t.is_contiguous()):
        raise ValueError(f"{name} must be contiguous float32 {(H,)} on {like.device}")
    return t


def _scale(scale: Optional[float], dk: int, lam: Optional[torch.Tensor]) -> float:
    return (dk if lam is None else dk / 2) ** -0.5 if scale is None else float(scale)


def _head_strides(*tensors):
    """ret_strides of tensors of three or four dimensions in the order of their shape, or NULL when all are contiguous."""
    if all(t.is_contiguous() for t in tensors):
        return None
    return _pack(*((t.stride(0), t.stride(1), t.stride(2) if t.dim() == 4 else 0) for t in tensors))


def _qkv(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, dims: int):
    if q.dim() != dims or k.dim() != dims or v.dim() != dims:
        raise ValueError("expected q [B,H,T,dk], k [B,Hk,S,dk], v [B,Hk,S,dv]" if dims == 4 else
                         "expected q [B,H,dk], k [B,Hk,dk], v [B,Hk,dv]")
    dt = _dtype(q)
    B, H, dk, dv = q.shape[0], q.shape[1], q.shape[-1], v.shape[-1]
    inner = k.shape[1:-1]
    _sizes(*q.shape, *k.shape, dv)
    _rows(q, q.shape, q, "q")
    _rows(k, (B, *inner, dk), q, "k")
    _rows(v, (B, *inner, dv), q, "v")
    return dt, B, H, k.shape[1], dk, dv


def _mask(causal: bool, offset: Optional[int], T: int, S: int) -> Tuple[int, int]:
    off = (S - T if offset is None else int(offset)) if causal else 0
    _sizes(off)
    return int(bool(causal)), off


def attention_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, lam: Optional[torch.Tensor] = None,
                  causal: bool = True, scale: Optional[float] = None, offset: Optional[int] = None,
                  lens: Optional[torch.Tensor] = None, keep: bool = False, o: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None
                  ) -> Union[torch.Tensor, Tuple[torch.Tensor, Tuple[torch.Tensor, Optional[torch.Tensor]]]]:
    """Softmax attention over a whole sequence (retention_attention_fwd).

    q [B,H,T,dk]; k [B,Hk,S,dk], v [B,Hk,S,dv] with H a multiple of Hk (float32 or bfloat16; rows contiguous,
    any other strides).  lam: optional float32 [H]: differential attention, the map of the first half of the dk
    channels less lam times the map of the second half.  causal: row t sees the keys up to t + offset (default
    S - T); lens: optional int32 [B], keys of each sequence.  scale: default 1 / sqrt(channels of a map).
    Rows that see no key are 0.  Returns o [B,H,T,dv], and with keep (o, kept) for attention_bwd.
    """
    lib = load()
    dt, B, H, Hk, dk, dv = _qkv(q, k, v, 4)
    T, S = q.shape[2], k.shape[2]
    _weights(lam, H, q, "lam")
    _i32(lens, (B,), q, "lens")
    maps = 1 if lam is None else 2
    o = torch.empty((B, H, T, dv), dtype=q.dtype, device=q.device) if o is None else _rows(o, (B, H, T, dv), q, "o")
    lse = second = None
    if keep:
        lse = torch.empty((B, H, maps, T), dtype=torch.float32, device=q.device)
        second = torch.empty((B, H, T, dv), dtype=q.dtype, device=q.device) if maps > 1 else None
    on, off = _mask(causal, offset, T, S)
    ws, wp, wn = _workspace(workspace, lib.retention_attention_workspace_bytes(B, H, Hk, T, S, dk, dv, maps, dt), q)
    _call(lib.retention_attention_fwd, q.device, q.data_ptr(), k.data_ptr(), v.data_ptr(), _p(lam), _p(lens),
          o.data_ptr(), _p(lse), _p(second), _head_strides(q, k, v, o), B, H, Hk, T, S, dk, dv, _scale(scale, dk, lam),
          on, off, dt, wp, wn)
    return (o, (lse, second)) if keep else o


def attention_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor, grad_o: torch.Tensor, kept,
                  lam: Optional[torch.Tensor] = None, causal: bool = True, scale: Optional[float] = None,
                  offset: Optional[int] = None, lens: Optional[torch.Tensor] = None,
                  grad_q: Optional[torch.Tensor] = None, grad_k: Optional[torch.Tensor] = None,
                  grad_v: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None
                  ) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor, Optional[torch.Tensor]]:
    """Gradients of attention_fwd (retention_attention_bwd): (grad_q, grad_k, grad_v, grad_lam).

    o and kept: what the forward call with keep=True returned; lam, causal, scale, offset, lens: that call's.
    grad_lam (float32 [H]) is None without lam.
    """
    lib = load()
    dt, B, H, Hk, dk, dv = _qkv(q, k, v, 4)
    T, S = q.shape[2], k.shape[2]
    _weights(lam, H, q, "lam")
    _i32(lens, (B,), q, "lens")
    maps = 1 if lam is None else 2
    _rows(o, (B, H, T, dv), q, "o")
    _rows(grad_o, (B, H, T, dv), q, "grad_o")
    lse, second = kept
    if (lse.dtype != torch.float32 or lse.shape != (B, H, maps, T) or lse.get_device() != q.get_device() or
            not lse.is_contiguous()):
        raise ValueError(f"kept must come from attention_fwd with the same arguments (lse {(B, H, maps, T)})")
    if (second is not None) != (lam is not None):
        raise ValueError("kept must come from attention_fwd with the same lam")
    if second is not None and not _rows(second, (B, H, T, dv), q, "kept[1]").is_contiguous():
        raise ValueError("kept[1] must be contiguous")
    gq, gk, gv = _out(grad_q, q, "grad_q"), _out(grad_k, k, "grad_k"), _out(grad_v, v, "grad_v")
    glam = None if lam is None else torch.empty_like(lam)
    on, off = _mask(causal, offset, T, S)
    ws, wp, wn = _workspace(workspace, lib.retention_attention_bwd_workspace_bytes(B, H, Hk, T, S, dk, dv, maps, dt), q)
    _call(lib.retention_attention_bwd, q.device, q.data_ptr(), k.data_ptr(), v.data_ptr(), _p(lam), _p(lens),
          o.data_ptr(), lse.data_ptr(), _p(second), grad_o.data_ptr(), gq.data_ptr(), gk.data_ptr(), gv.data_ptr(),
          _p(glam), _head_strides(q, k, v, o, grad_o, gq, gk, gv), B, H, Hk, T, S, dk, dv, _scale(scale, dk, lam), on,
          off, dt, wp, wn)
    return gq, gk, gv, glam


def _cache(k_cache: torch.Tensor, v_cache: torch.Tensor, table: torch.Tensor, like: torch.Tensor, B: int, Hk: int,
           dk: int, dv: int):
    if k_cache.dim() != 4 or v_cache.dim() != 4:
        raise ValueError("expected k_cache [pages,Hk,page,dk] and v_cache [pages,Hk,page,dv]")
    pages, page = k_cache.shape[0], k_cache.shape[2]
    _rows(k_cache, (pages, Hk, page, dk), like, "k_cache")
    _rows(v_cache, (pages, Hk, page, dv), like, "v_cache")
    if table.dim() != 2:
        raise ValueError("expected table [B,max_pages]")
    _i32(table, (B, table.shape[1]), like, "table")
    return _sizes(pages, page, table.shape[1])


def attention_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                   table: torch.Tensor, lens: torch.Tensor, lam: Optional[torch.Tensor] = None,
                   scale: Optional[float] = None, o: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Attention of one new token of every sequence, in place on a paged cache (retention_attention_step).

    q [B,H,dk]; k [B,Hk,dk], v [B,Hk,dv]: stored as token lens[b] of the sequence, which q sees with all tokens
    before it.  k_cache [pages,Hk,page,dk], v_cache [pages,Hk,page,dv]; table int32 [B,max_pages]: the pages of
    each sequence in order (a number outside 0..pages-1: none); lens int32 [B], tokens in the cache before the
    call (negative: an idle sequence, o is 0).  lens is not advanced.  lam, scale: as in attention_fwd.
    Returns o [B,H,dv].
    """
    lib = load()
    dt, B, H, Hk, dk, dv = _qkv(q, k, v, 3)
    pages, page, most = _cache(k_cache, v_cache, table, q, B, Hk, dk, dv)
    if lens is None:
        raise ValueError("lens is required")
    _i32(lens, (B,), q, "lens")
    _weights(lam, H, q, "lam")
    maps = 1 if lam is None else 2
    o = torch.empty((B, H, dv), dtype=q.dtype, device=q.device) if o is None else _rows(o, (B, H, dv), q, "o")
    ws, wp, wn = _workspace(
        workspace, lib.retention_attention_step_workspace_bytes(B, H, Hk, dk, dv, page, most, maps, dt), q)
    _call(lib.retention_attention_step, q.device, q.data_ptr(), k.data_ptr(), v.data_ptr(), k_cache.data_ptr(),
          v_cache.data_ptr(), table.data_ptr(), lens.data_ptr(), _p(lam), o.data_ptr(),
          _head_strides(q, k, v, k_cache, v_cache, o), B, H, Hk, dk, dv, pages, page, most, _scale(scale, dk, lam), dt,
          wp, wn)
    return o


def cache_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, table: torch.Tensor,
                 start: torch.Tensor, counts: Optional[torch.Tensor] = None) -> None:
    """Stores keys and values of T tokens of every sequence in a paged cache (retention_cache_append).

    k [B,Hk,T,dk], v [B,Hk,T,dv]; token t < counts[b] (default T) of sequence b becomes its token start[b] + t.
    k_cache, v_cache, table: as in attention_step; start, counts: int32 [B] (a negative start: an idle sequence).
    """
    if k.dim() != 4 or v.dim() != 4:
        raise ValueError("expected k [B,Hk,T,dk] and v [B,Hk,T,dv]")
    dt = _dtype(k)
    B, Hk, T, dk = _sizes(*k.shape)
    dv = v.shape[-1]
    _rows(k, k.shape, k, "k")
    _rows(v, (B, Hk, T, dv), k, "v")
    pages, page, most = _cache(k_cache, v_cache, table, k, B, Hk, dk, dv)
    if start is None:
        raise ValueError("start is required")
    _i32(start, (B,), k, "start")
    _i32(counts, (B,), k, "counts")
    _call(load().retention_cache_append, k.device, k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
          table.data_ptr(), start.data_ptr(), _p(counts), _head_strides(k, v, k_cache, v_cache), B, Hk, T, dk, dv, pages,
          page, most, dt)

"""ctypes binding of the attention calls: ordinary and differential softmax
attention over whole sequences, its gradients, the decode step over a paged
cache, and the cache's filling.

As in _block, this is argument marshalling only, and sequence tensors and caches
may have any strides as long as the elements of a row are contiguous.
"""
from __future__ import annotations

from functools import lru_cache
from typing import Optional, Tuple, Union

import torch

from ._block import _BAD, _call, _dtype, _out, _p, _pack, _raw_stream, _rows, _workspace
from ._lib import RetentionError, _sizes, last_error, load

# A decode step's kernel takes as long as this module's checks, so they ask each
# tensor once: _seq, _launch and _bytes are quicker forms of _rows, _call and the
# library's workspace queries.
_get_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device
_MOST = 0x7FFFFFFF


def _seq(t: torch.Tensor, shape, dtype: torch.dtype, dev: int, like: torch.Tensor, name: str) -> bool:
    """_rows(t, shape, like, name) for like's dtype and device number; whether t is contiguous."""
    if t.shape == shape and t.dtype == dtype and t.get_device() == dev and dev >= 0 and t.is_contiguous():
        return True
    return _rows(t, shape, like, name).is_contiguous()


def _launch(fn, dev: int, like: torch.Tensor, *args) -> None:
    if _raw_stream is None or dev != _get_device():
        return _call(fn, like.device, *args)
    st = fn(*args, _raw_stream(dev))
    if st != 0:
        raise RetentionError(st, last_error())


@lru_cache(maxsize=1024)
def _bytes(call: str, *sizes: int) -> int:
    """Workspace of a call of these sizes; what the library refuses is raised, and not kept."""
    need = getattr(load(), call)(*sizes)
    if need == _BAD:
        raise RetentionError(1, last_error())
    return need


def _i32(t: Optional[torch.Tensor], shape, dev: int, like: torch.Tensor, name: str) -> Optional[torch.Tensor]:
    """Lengths, positions or page numbers: contiguous int32 on the same device."""
    if t is not None and (t.dtype != torch.int32 or t.shape != shape or t.get_device() != dev or
                          not t.is_contiguous()):
        raise ValueError(f"{name} must be contiguous int32 {tuple(shape)} on {like.device}")
    return t


def _weights(t: Optional[torch.Tensor], H: int, dev: int, like: torch.Tensor, name: str) -> Optional[torch.Tensor]:
    if t is not None and (t.dtype != torch.float32 or t.shape != (H,) or t.get_device() != dev or
                          not t.is_contiguous()):
        raise ValueError(f"{name} must be contiguous float32 {(H,)} on {like.device}")
    return t


def _scale(scale: Optional[float], dk: int, lam: Optional[torch.Tensor]) -> float:
    return (dk if lam is None else dk / 2) ** -0.5 if scale is None else float(scale)


def _head_strides(*tensors):
    """ret_strides of tensors of three or four dimensions in the order of their shape."""
    return _pack(*((t.stride(0), t.stride(1), t.stride(2) if t.dim() == 4 else 0) for t in tensors))


def _qkv(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, dims: int):
    """(dtype code, device number, all contiguous, B, H, Hk, dk, dv)."""
    qs, ks, vs = q.shape, k.shape, v.shape
    if len(qs) != dims or len(ks) != dims or len(vs) != dims:
        raise ValueError("expected q [B,H,T,dk], k [B,Hk,S,dk], v [B,Hk,S,dv]" if dims == 4 else
                         "expected q [B,H,dk], k [B,Hk,dk], v [B,Hk,dv]")
    dt, dtype, dev = _dtype(q), q.dtype, q.get_device()
    B, H, Hk, dk, dv = qs[0], qs[1], ks[1], qs[-1], vs[-1]
    if not (0 < q.numel() <= _MOST and 0 < k.numel() <= _MOST and 0 < v.numel() <= _MOST):
        _sizes(*qs, *ks, dv)  # the element counts tell most tensors fit
    flat = _seq(q, qs, dtype, dev, q, "q")
    flat &= _seq(k, (B, *ks[1:-1], dk), dtype, dev, q, "k")
    flat &= _seq(v, (B, *ks[1:-1], dv), dtype, dev, q, "v")
    return dt, dev, flat, B, H, Hk, dk, dv


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
    dt, dev, flat, B, H, Hk, dk, dv = _qkv(q, k, v, 4)
    T, S = q.shape[2], k.shape[2]
    _weights(lam, H, dev, q, "lam")
    _i32(lens, (B,), dev, q, "lens")
    maps = 1 if lam is None else 2
    if o is None:
        o = q.new_empty((B, H, T, dv))
    else:
        flat &= _seq(o, (B, H, T, dv), q.dtype, dev, q, "o")
    lse = second = None
    if keep:
        lse = q.new_empty((B, H, maps, T), dtype=torch.float32)
        second = q.new_empty((B, H, T, dv)) if maps > 1 else None
    on, off = _mask(causal, offset, T, S)
    ws, wp, wn = _workspace(workspace, _bytes("retention_attention_workspace_bytes", B, H, Hk, T, S, dk, dv, maps, dt), q)
    _launch(load().retention_attention_fwd, dev, q, q.data_ptr(), k.data_ptr(), v.data_ptr(), _p(lam), _p(lens),
          o.data_ptr(), _p(lse), _p(second), None if flat else _head_strides(q, k, v, o), B, H, Hk, T, S, dk, dv, _scale(scale, dk, lam),
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
    dt, dev, flat, B, H, Hk, dk, dv = _qkv(q, k, v, 4)
    T, S = q.shape[2], k.shape[2]
    _weights(lam, H, dev, q, "lam")
    _i32(lens, (B,), dev, q, "lens")
    maps = 1 if lam is None else 2
    flat &= _seq(o, (B, H, T, dv), q.dtype, dev, q, "o")
    flat &= _seq(grad_o, (B, H, T, dv), q.dtype, dev, q, "grad_o")
    lse, second = kept
    if (lse.dtype != torch.float32 or lse.shape != (B, H, maps, T) or lse.get_device() != dev or
            not lse.is_contiguous()):
        raise ValueError(f"kept must come from attention_fwd with the same arguments (lse {(B, H, maps, T)})")
    if (second is not None) != (lam is not None):
        raise ValueError("kept must come from attention_fwd with the same lam")
    if second is not None and not _seq(second, (B, H, T, dv), q.dtype, dev, q, "kept[1]"):
        raise ValueError("kept[1] must be contiguous")
    gq, gk, gv = _out(grad_q, q, "grad_q"), _out(grad_k, k, "grad_k"), _out(grad_v, v, "grad_v")
    flat = flat and gq.is_contiguous() and gk.is_contiguous() and gv.is_contiguous()
    glam = None if lam is None else torch.empty_like(lam)
    on, off = _mask(causal, offset, T, S)
    ws, wp, wn = _workspace(workspace, _bytes("retention_attention_bwd_workspace_bytes", B, H, Hk, T, S, dk, dv, maps, dt), q)
    _launch(load().retention_attention_bwd, dev, q, q.data_ptr(), k.data_ptr(), v.data_ptr(), _p(lam), _p(lens),
          o.data_ptr(), lse.data_ptr(), _p(second), grad_o.data_ptr(), gq.data_ptr(), gk.data_ptr(), gv.data_ptr(),
          _p(glam), None if flat else _head_strides(q, k, v, o, grad_o, gq, gk, gv), B, H, Hk, T, S, dk, dv, _scale(scale, dk, lam), on,
          off, dt, wp, wn)
    return gq, gk, gv, glam


def _cache(k_cache: torch.Tensor, v_cache: torch.Tensor, table: torch.Tensor, dev: int, like: torch.Tensor, B: int,
           Hk: int, dk: int, dv: int):
    """(both contiguous, pages, tokens of a page, pages of a sequence)."""
    ks = k_cache.shape
    if len(ks) != 4 or v_cache.dim() != 4:
        raise ValueError("expected k_cache [pages,Hk,page,dk] and v_cache [pages,Hk,page,dv]")
    pages, page = ks[0], ks[2]
    flat = _seq(k_cache, (pages, Hk, page, dk), like.dtype, dev, like, "k_cache")
    flat &= _seq(v_cache, (pages, Hk, page, dv), like.dtype, dev, like, "v_cache")
    if table.dim() != 2:
        raise ValueError("expected table [B,max_pages]")
    most = table.shape[1]
    _i32(table, (B, most), dev, like, "table")
    if pages > _MOST or page > _MOST or most > _MOST:
        _sizes(pages, page, most)
    return flat, pages, page, most


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
    dt, dev, flat, B, H, Hk, dk, dv = _qkv(q, k, v, 3)
    rows_flat, pages, page, most = _cache(k_cache, v_cache, table, dev, q, B, Hk, dk, dv)
    flat &= rows_flat
    if lens is None:
        raise ValueError("lens is required")
    _i32(lens, (B,), dev, q, "lens")
    _weights(lam, H, dev, q, "lam")
    maps = 1 if lam is None else 2
    if o is None:
        o = q.new_empty((B, H, dv))
    else:
        flat &= _seq(o, (B, H, dv), q.dtype, dev, q, "o")
    ws, wp, wn = _workspace(
        workspace, _bytes("retention_attention_step_workspace_bytes", B, H, Hk, dk, dv, page, most, maps, dt), q)
    _launch(load().retention_attention_step, dev, q, q.data_ptr(), k.data_ptr(), v.data_ptr(), k_cache.data_ptr(),
          v_cache.data_ptr(), table.data_ptr(), lens.data_ptr(), _p(lam), o.data_ptr(),
          None if flat else _head_strides(q, k, v, k_cache, v_cache, o), B, H, Hk, dk, dv, pages, page, most, _scale(scale, dk, lam), dt,
          wp, wn)
    return o


def cache_append(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, table: torch.Tensor,
                 start: torch.Tensor, counts: Optional[torch.Tensor] = None) -> None:
    """Stores keys and values of T tokens of every sequence in a paged cache (retention_cache_append).

    k [B,Hk,T,dk], v [B,Hk,T,dv]; token t < counts[b] (default T) of sequence b becomes its token start[b] + t.
    k_cache, v_cache, table: as in attention_step; start, counts: int32 [B] (a negative start: an idle sequence).
    """
    ks = k.shape
    if len(ks) != 4 or v.dim() != 4:
        raise ValueError("expected k [B,Hk,T,dk] and v [B,Hk,T,dv]")
    dt, dtype, dev = _dtype(k), k.dtype, k.get_device()
    if not 0 < k.numel() <= _MOST:
        _sizes(*ks)
    B, Hk, T, dk = ks
    dv = v.shape[-1]
    flat = _seq(k, ks, dtype, dev, k, "k")
    flat &= _seq(v, (B, Hk, T, dv), dtype, dev, k, "v")
    rows_flat, pages, page, most = _cache(k_cache, v_cache, table, dev, k, B, Hk, dk, dv)
    flat &= rows_flat
    if start is None:
        raise ValueError("start is required")
    _i32(start, (B,), dev, k, "start")
    _i32(counts, (B,), dev, k, "counts")
    _launch(load().retention_cache_append, dev, k, k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
          table.data_ptr(), start.data_ptr(), _p(counts), None if flat else _head_strides(k, v, k_cache, v_cache), B, Hk, T, dk, dv, pages,
          page, most, dt)

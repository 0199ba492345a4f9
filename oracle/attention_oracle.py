"""fp64 CPU oracle of softmax attention, ordinary and differential, its
gradients by the chain rule, and a decode step over a paged cache.  Plain
torch-CPU code written from the formulas, head by head; shares no code with the
HIP path.
"""
from __future__ import annotations

from typing import Optional

import torch

F64 = torch.float64


def _up(t: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    return None if t is None else t.detach().to("cpu", F64)


def visible(T: int, S: int, length: int, causal: bool, offset: int) -> torch.Tensor:
    """[T,S]: whether row t sees key s."""
    s, t = torch.arange(S)[None, :], torch.arange(T)[:, None]
    m = (s < length).expand(T, S)
    return m & (s <= t + offset) if causal else m


def _map(q, k, scale, m):
    """(A, lse) of one map of one head; rows that see no key are 0 and -inf."""
    x = (scale * (q @ k.T)).masked_fill(~m, -torch.inf)
    top = x.amax(-1, keepdim=True) if x.shape[-1] else torch.full((x.shape[0], 1), -torch.inf, dtype=F64)
    e = torch.exp(x - torch.where(top == -torch.inf, torch.zeros_like(top), top))
    e = torch.where(m, e, torch.zeros_like(e))
    z = e.sum(-1, keepdim=True)
    return e / torch.where(z == 0, torch.ones_like(z), z), (top + torch.log(z)).squeeze(-1)


def _heads(q, k, v, lam, causal, scale, offset, lens):
    """Every (b, h): (b, h, hk, q, k, v, per-map slices, visible)."""
    B, H, T, dk = q.shape
    Hk, S = k.shape[1], k.shape[2]
    maps = 1 if lam is None else 2
    d = dk // maps
    scale = d ** -0.5 if scale is None else scale
    offset = S - T if offset is None else offset
    for b in range(B):
        n = S if lens is None else min(max(int(lens[b]), 0), S)
        m = visible(T, S, n, causal, offset)
        vv = [torch.where(torch.arange(S)[:, None] < n, x[b], torch.zeros((), dtype=F64)) for x in (k, v)]
        for h in range(H):
            hk = h // (H // Hk)
            yield b, h, hk, q[b, h], vv[0][hk], vv[1][hk], [slice(i * d, (i + 1) * d) for i in range(maps)], scale, m


def attention(q, k, v, lam=None, causal: bool = True, scale=None, offset=None, lens=None):
    """(o [B,H,T,dv], lse [B,H,maps,T], second [B,H,T,dv] or None)."""
    q, k, v, lam = _up(q), _up(k), _up(v), _up(lam)
    o = torch.zeros(*q.shape[:3], v.shape[-1], dtype=F64)
    lse = torch.zeros(q.shape[0], q.shape[1], 1 if lam is None else 2, q.shape[2], dtype=F64)
    second = None if lam is None else torch.zeros_like(o)
    for b, h, _, qq, kk, vv, parts, sc, m in _heads(q, k, v, lam, causal, scale, offset, lens):
        for i, p in enumerate(parts):
            A, lse[b, h, i] = _map(qq[:, p], kk[:, p], sc, m)
            y = A @ vv
            o[b, h] += y if i == 0 else -lam[h] * y
            if i == 1:
                second[b, h] = y
    return o, lse, second


def attention_backward(q, k, v, grad_o, lam=None, causal: bool = True, scale=None, offset=None, lens=None):
    """(grad_q, grad_k, grad_v, grad_lam) for L = sum <grad_o, o>."""
    q, k, v, lam, do = _up(q), _up(k), _up(v), _up(lam), _up(grad_o)
    gq, gk, gv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    gl = None if lam is None else torch.zeros_like(lam)
    for b, h, hk, qq, kk, vv, parts, sc, m in _heads(q, k, v, lam, causal, scale, offset, lens):
        dA = do[b, h] @ vv.T
        for i, p in enumerate(parts):
            w = 1.0 if i == 0 else -float(lam[h])
            A, _ = _map(qq[:, p], kk[:, p], sc, m)
            mean = (A * dA).sum(-1, keepdim=True)
            dx = w * A * (dA - mean)
            gq[b, h][:, p] += sc * dx @ kk[:, p]
            gk[b, hk][:, p] += sc * dx.T @ qq[:, p]
            gv[b, hk] += w * A.T @ do[b, h]
            if i == 1:
                gl[h] -= mean.sum()
    return gq, gk, gv, gl


def _page(table, b, s, page, pages):
    p = int(table[b, s // page])
    return p if 0 <= p < pages else None


def cache_append(k, v, k_cache, v_cache, table, start, counts=None):
    """The caches after the call (copies, in their type)."""
    kc, vc = k_cache.clone(), v_cache.clone()
    pages, page, most = kc.shape[0], kc.shape[2], table.shape[1]
    for b in range(k.shape[0]):
        n = k.shape[2] if counts is None else min(int(counts[b]), k.shape[2])
        for t in range(n):
            s = int(start[b]) + t
            if int(start[b]) < 0 or s >= most * page:
                continue
            p = _page(table, b, s, page, pages)
            if p is not None:
                kc[p, :, s % page], vc[p, :, s % page] = k[b, :, t], v[b, :, t]
    return kc, vc


def attention_step(q, k, v, k_cache, v_cache, table, lens, lam=None, scale=None):
    """(o [B,H,dv], k_cache, v_cache after the call)."""
    o = torch.zeros(*q.shape[:2], v.shape[-1], dtype=F64)
    pages, page, most = k_cache.shape[0], k_cache.shape[2], table.shape[1]
    for b in range(q.shape[0]):
        n = int(lens[b])
        if n < 0:
            continue
        at = [(p, s % page) for s in range(min(n, most * page)) for p in [_page(table, b, s, page, pages)] if p is not None]
        ks = torch.stack([k_cache[p, :, r] for p, r in at] + [k[b]], 1)[None]
        vs = torch.stack([v_cache[p, :, r] for p, r in at] + [v[b]], 1)[None]
        o[b] = attention(q[b:b + 1, :, None], ks, vs, lam, False, scale)[0][0, :, 0]
    kc, vc = cache_append(k[:, :, None], v[:, :, None], k_cache, v_cache, table, lens)
    return o, kc, vc

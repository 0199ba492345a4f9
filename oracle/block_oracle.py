"""fp64 CPU oracle of the operators around retention in a block: the gated
scan, the gated per-head GroupNorm and the residual norm, each with its
gradient by the chain rule.  Plain torch-CPU code written from the formulas;
shares no code with the HIP path.
"""
from __future__ import annotations

from typing import Optional, Sequence, Tuple

import torch

F64 = torch.float64


def _up(t: Optional[torch.Tensor]) -> Optional[torch.Tensor]:
    return None if t is None else t.detach().to("cpu", F64)


# ------------------------------------------------------------- gated scan
def _log_decay(f: torch.Tensor, rate: Sequence[float]) -> torch.Tensor:
    """rate_h log sigmoid(f) for f [B,H,...]; rates are rounded to fp32 as the library takes them."""
    r = torch.tensor([float(x) for x in rate], dtype=torch.float32).to(F64)
    return r.view(1, -1, *([1] * (f.dim() - 2))) * -torch.logaddexp(torch.zeros_like(f), -f)


def gated_scan(x, f, rate, state_in=None, normalize: bool = False) -> Tuple[torch.Tensor, torch.Tensor]:
    """h_t = a_t h_(t-1) + u_t, one token at a time: (h [B,H,T,d], last h [B,H,d])."""
    x, f, s = _up(x), _up(f), _up(state_in)
    B, H, T, d = x.shape
    z = _log_decay(f, rate)
    h = torch.zeros(B, H, d, dtype=F64) if s is None else s
    out = torch.empty_like(x)
    for t in range(T):
        a = torch.exp(z[:, :, t])
        u = -torch.expm1(z[:, :, t]) * x[:, :, t] if normalize else x[:, :, t]
        h = a * h + u
        out[:, :, t] = h
    return out, h


def gated_scan_backward(x, f, rate, grad_y, state_in=None, grad_state_out=None, normalize: bool = False):
    """(grad_x, grad_f, grad_state_in) for L = sum <grad_y, y> + <grad_state_out, state_out>."""
    h, _ = gated_scan(x, f, rate, state_in, normalize)
    x, f, dy, s, ds = _up(x), _up(f), _up(grad_y), _up(state_in), _up(grad_state_out)
    B, H, T, d = x.shape
    r = torch.tensor([float(v) for v in rate], dtype=torch.float32).to(F64).view(1, -1, 1)
    z = _log_decay(f, rate)
    later = torch.zeros(B, H, d, dtype=F64) if ds is None else ds
    gx, gf = torch.empty_like(x), torch.empty_like(x)
    for t in range(T - 1, -1, -1):
        g = dy[:, :, t] + later
        a, c = torch.exp(z[:, :, t]), -torch.expm1(z[:, :, t])
        before = h[:, :, t - 1] if t > 0 else (torch.zeros_like(g) if s is None else s)
        da = g * (before - x[:, :, t]) if normalize else g * before
        gx[:, :, t] = g * c if normalize else g
        gf[:, :, t] = da * a * r * torch.sigmoid(-f[:, :, t])
        later = a * g
    return gx, gf, later


# ----------------------------------------------------------- gated GroupNorm
def _normalised(y: torch.Tensor, eps: float, center: bool):
    mu = y.mean(-1, keepdim=True) if center else torch.zeros_like(y[..., :1])
    rstd = 1.0 / torch.sqrt(((y - mu) ** 2).mean(-1, keepdim=True) + eps)
    return (y - mu) * rstd, rstd


def _norm_backward(xh, rstd, p, center: bool):
    """d/dy of sum <p, xh(y)>."""
    t = p - xh * (p * xh).mean(-1, keepdim=True)
    if center:
        t = t - p.mean(-1, keepdim=True)
    return rstd * t


def group_norm_gated(y, gate=None, weight=None, bias=None, eps: float = 1e-5) -> torch.Tensor:
    """Per-head GroupNorm of y [B,H,T,dv] times gate sigmoid(gate), gate and result [B,T,H,dv]."""
    y, z, w, b = _up(y), _up(gate), _up(weight), _up(bias)
    n, _ = _normalised(y, eps, True)
    n = n if w is None else n * w[:, None]
    n = (n if b is None else n + b[:, None]).transpose(1, 2)
    return n if z is None else n * z * torch.sigmoid(z)


def group_norm_gated_backward(y, gate, grad_out, weight=None, bias=None, eps: float = 1e-5):
    """(grad_y, grad_gate, grad_weight, grad_bias); grad_gate None without a gate."""
    y, z, do, w, b = _up(y), _up(gate), _up(grad_out), _up(weight), _up(bias)
    xh, rstd = _normalised(y, eps, True)
    n = xh if w is None else xh * w[:, None]
    n = n if b is None else n + b[:, None]
    dz = None
    dn = do.transpose(1, 2)
    if z is not None:
        zt = z.transpose(1, 2)
        s = torch.sigmoid(zt)
        dz = (dn * n * (s + zt * s * (1 - s))).transpose(1, 2)
        dn = dn * zt * s
    p = dn if w is None else dn * w[:, None]
    return _norm_backward(xh, rstd, p, True), dz, (dn * xh).sum((0, 2)), dn.sum((0, 2))


# ------------------------------------------------------------- residual norm
def residual(x, f, scale=None, alpha: float = 1.0) -> torch.Tensor:
    """The stream alpha x + scale f before it is rounded to its type."""
    x, f, s = _up(x), _up(f), _up(scale)
    return alpha * x + (f if s is None else s * f)


def stream_norm(r, weight=None, bias=None, eps: float = 1e-5, rms: bool = False) -> torch.Tensor:
    """LayerNorm or RMSNorm of the stored stream r over its last dimension."""
    n, _ = _normalised(_up(r), eps, not rms)
    w, b = _up(weight), _up(bias)
    n = n if w is None else n * w
    return n if b is None else n + b


def residual_norm_backward(r, grad_n, grad_r=None, weight=None, f=None, scale=None, alpha: float = 1.0,
                           eps: float = 1e-5, rms: bool = False):
    """(grad_x, grad_f, grad_weight, grad_bias, grad_scale) from the stored r."""
    r, dn, dr, w, f, s = _up(r), _up(grad_n), _up(grad_r), _up(weight), _up(f), _up(scale)
    xh, rstd = _normalised(r, eps, not rms)
    g = _norm_backward(xh, rstd, dn if w is None else dn * w, not rms)
    g = g if dr is None else g + dr
    rows = tuple(range(r.dim() - 1))
    gs = None if s is None or f is None else (g * f).sum(rows)
    return alpha * g, g if s is None else s * g, (dn * xh).sum(rows), dn.sum(rows), gs

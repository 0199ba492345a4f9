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

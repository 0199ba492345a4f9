"""ctypes binding of the operators around retention in a block: the gated scan,
the gated per-head GroupNorm and the residual norm.

As in _lib, this is argument marshalling only: tensors are checked for device,
dtype and shape, and their pointers, strides and the current stream of their
device go through the C ABI.  Sequence tensors may have any strides as long as
the elements of a row are contiguous (token-major tensors, slices of a fused
projection).
"""
from __future__ import annotations

import ctypes
from typing import Optional, Tuple, Union

import torch

from ._lib import RET_BF16, RET_F32, RetentionError, _gamma_array, _shape, _sizes, last_error, load

_DT = {torch.float32: RET_F32, torch.bfloat16: RET_BF16}
_BAD = ctypes.c_size_t(-1).value
_current_device = torch.cuda.current_device
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else None


def _dtype(t: torch.Tensor) -> int:
    dt = _DT.get(t.dtype)
    if dt is None:
        raise TypeError(f"unsupported dtype {t.dtype}; use float32 or bfloat16")
    return dt


def _rows(t: torch.Tensor, shape, like: torch.Tensor, name: str) -> torch.Tensor:
    """A sequence tensor: shape, dtype and device, and contiguous rows."""
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.dtype != like.dtype or t.get_device() != like.get_device() or not t.is_cuda:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a device (cuda/HIP) tensor")
        raise ValueError(f"{name} must be {like.dtype} on {like.device}, got {t.dtype} on {t.device}")
    if not t.is_contiguous() and t.stride(-1) != 1 and t.shape[-1] > 1:
        raise ValueError(f"the rows (last dimension) of {name} must be contiguous")
    return t


def _f32(t: Optional[torch.Tensor], shape, like: torch.Tensor, name: str) -> Optional[torch.Tensor]:
    """A state or parameter: contiguous fp32 on the same device."""
    if t is not None and (t.dtype != torch.float32 or t.shape != shape or t.get_device() != like.get_device() or
                          not t.is_contiguous()):
        raise ValueError(f"{name} must be contiguous float32 {tuple(shape)} on {like.device}")
    return t


def _like(t: torch.Tensor) -> torch.Tensor:
    """A new contiguous tensor of t's shape and type."""
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def _new_f32(t: Union[torch.Tensor, bool, None], shape, like: torch.Tensor, name: str) -> Optional[torch.Tensor]:
    """An fp32 output: a tensor to fill, True for a new one, False or None for none."""
    if t is True:
        return torch.empty(shape, dtype=torch.float32, device=like.device)
    if t is None or t is False:
        return None
    return _f32(t, shape, like, name)


def _strides(*tensors):
    """ret_strides of [n0,n1,n2,row] tensors in the order of their shape, or NULL when all are contiguous."""
    if all(t.is_contiguous() for t in tensors):
        return None
    return (ctypes.c_longlong * (3 * len(tensors)))(*(s for t in tensors for s in t.stride()[:3]))


def _strides_bh(*tensors):
    """The same for one-token tensors [B,H,row]."""
    if all(t.is_contiguous() for t in tensors):
        return None
    return (ctypes.c_longlong * (3 * len(tensors)))(*(s for t in tensors for s in (t.stride(0), t.stride(1), 0)))


def _p(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _workspace(t: Optional[torch.Tensor], need: int, like: torch.Tensor):
    """(tensor, pointer, bytes) of a call's scratch; allocated on the current stream when none is given."""
    if need == _BAD:
        raise RetentionError(1, last_error())
    if t is None:
        if need == 0:
            return None, None, 0
        t = torch.empty(need, dtype=torch.uint8, device=like.device)
    elif t.device != like.device or not t.is_contiguous():
        raise ValueError(f"workspace must be contiguous on {like.device}")
    return t, t.data_ptr(), t.numel() * t.element_size()


def _call(fn, device: torch.device, *args) -> None:
    """fn(*args, stream) with the tensors' device current and on its current stream."""
    index = device.index
    if index != _current_device():
        with torch.cuda.device(device):
            st = fn(*args, torch.cuda.current_stream(device).cuda_stream)
    else:
        st = fn(*args, _raw_stream(index) if _raw_stream else torch.cuda.current_stream(device).cuda_stream)
    if st != 0:
        raise RetentionError(st, last_error())


def _out(t: Optional[torch.Tensor], like: torch.Tensor, name: str) -> torch.Tensor:
    return torch.empty_like(like) if t is None else _rows(t, like.shape, like, name)


def _scan_inputs(x: torch.Tensor, f: torch.Tensor, dims: int):
    if x.dim() != dims:
        raise ValueError("expected x and f [B,H,T,d]" if dims == 4 else "expected x and f [B,H,d]")
    if not 0 < x.numel() <= 0x7FFFFFFF:
        _sizes(*x.shape)
    dt = _dtype(x)
    _rows(x, x.shape, x, "x")
    _rows(f, x.shape, x, "f")
    return dt


def gated_scan_checkpoint_shape(B: int, H: int, T: int, d: int) -> Tuple[int, int, int, int]:
    """Shape of the fp32 checkpoints of a [B,H,T,d] call: the state before every block of tokens."""
    n = int(load().retention_gated_scan_checkpoint_bytes(*_sizes(B, H, T, d)))
    if n == _BAD:
        raise RetentionError(1, last_error())
    return B, H, n // (4 * B * H * d), d


def gated_scan_fwd(x: torch.Tensor, f: torch.Tensor, rate, state_in: Optional[torch.Tensor] = None,
                   state_out: Union[torch.Tensor, bool, None] = True, normalize: bool = False,
                   y: Optional[torch.Tensor] = None, checkpoints: Union[torch.Tensor, bool, None] = None,
                   workspace: Optional[torch.Tensor] = None):
    """Gated linear recurrence on the GPU (retention_gated_scan_fwd):
    h_t = a_t h_(t-1) + u_t, a_t = sigmoid(f_t)^rate_h, u_t = x_t or (normalize) (1 - a_t) x_t, y_t = h_t.

    x, f [B,H,T,d] (float32 or bfloat16; rows contiguous, any other strides); rate: H exponents > 0 on the
    host.  state_in: optional fp32 [B,H,d]; state_out: a tensor to fill (may be state_in), True to allocate
    one, False/None for none.  Returns (y, state_out), and with checkpoints (True, or a tensor of
    gated_scan_checkpoint_shape) (y, state_out, checkpoints) for gated_scan_bwd.
    """
    lib = load()
    dt = _scan_inputs(x, f, 4)
    B, H, T, d = x.shape
    state_in = _f32(state_in, (B, H, d), x, "state_in")
    state_out = _new_f32(state_out, (B, H, d), x, "state_out")
    y = _out(y, x, "y")
    want = checkpoints is not None and checkpoints is not False
    if want:
        checkpoints = _new_f32(checkpoints, gated_scan_checkpoint_shape(B, H, T, d), x, "checkpoints")
    else:
        checkpoints = None
    ws, wp, wn = _workspace(workspace, lib.retention_gated_scan_workspace_bytes(B, H, T, d, dt), x)
    _call(lib.retention_gated_scan_fwd, x.device, x.data_ptr(), f.data_ptr(), _gamma_array(rate, H), _p(state_in),
          _p(state_out), y.data_ptr(), _p(checkpoints), _strides(x, f, y), B, H, T, d, int(normalize), dt, wp, wn)
    return (y, state_out, checkpoints) if want else (y, state_out)


def gated_scan_bwd(x: torch.Tensor, f: torch.Tensor, rate, grad_y: torch.Tensor,
                   state_in: Optional[torch.Tensor] = None, grad_state_out: Optional[torch.Tensor] = None,
                   checkpoints: Optional[torch.Tensor] = None, normalize: bool = False,
                   grad_state_in: Union[torch.Tensor, bool, None] = True, grad_x: Optional[torch.Tensor] = None,
                   grad_f: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None
                   ) -> Tuple[torch.Tensor, torch.Tensor, Optional[torch.Tensor]]:
    """Gradients of gated_scan_fwd (retention_gated_scan_bwd): (grad_x, grad_f, grad_state_in).

    x, f, rate, state_in, normalize: the forward call's.  checkpoints: what that call returned; without them
    the forward recurrence is run again.  grad_state_in: a tensor to fill (may be grad_state_out), True to
    allocate one, False/None for none.
    """
    lib = load()
    dt = _scan_inputs(x, f, 4)
    B, H, T, d = x.shape
    _rows(grad_y, x.shape, x, "grad_y")
    vec = (B, H, d)
    state_in = _f32(state_in, vec, x, "state_in")
    grad_state_out = _f32(grad_state_out, vec, x, "grad_state_out")
    grad_state_in = _new_f32(grad_state_in, (B, H, d), x, "grad_state_in")
    if checkpoints is not None:
        _f32(checkpoints, gated_scan_checkpoint_shape(B, H, T, d), x, "checkpoints")
    gx = _out(grad_x, x, "grad_x")
    gf = _out(grad_f, x, "grad_f")
    ws, wp, wn = _workspace(workspace,
                            lib.retention_gated_scan_bwd_workspace_bytes(B, H, T, d, dt, checkpoints is not None), x)
    _call(lib.retention_gated_scan_bwd, x.device, x.data_ptr(), f.data_ptr(), _gamma_array(rate, H), _p(state_in),
          _p(checkpoints), grad_y.data_ptr(), _p(grad_state_out), gx.data_ptr(), gf.data_ptr(), _p(grad_state_in),
          _strides(x, f, grad_y, gx, gf), B, H, T, d, int(normalize), dt, wp, wn)
    return gx, gf, grad_state_in


def gated_scan_step(x: torch.Tensor, f: torch.Tensor, rate, state: torch.Tensor, normalize: bool = False,
                    y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One decode step of the gated recurrence (retention_gated_scan_step): state <- a state + u in place,
    returns y = state in the input dtype.  x, f [B,H,d]; state fp32 [B,H,d]."""
    dt = _scan_inputs(x, f, 3)
    B, H, d = x.shape
    if state is None:
        raise ValueError("state is required")
    _f32(state, x.shape, x, "state")
    y = _out(y, x, "y")
    _call(load().retention_gated_scan_step, x.device, x.data_ptr(), f.data_ptr(), _gamma_array(rate, H),
          state.data_ptr(), y.data_ptr(), _strides_bh(x, f, y), B, H, d, int(normalize), dt)
    return y


# ----------------------------------------------------------- gated GroupNorm
def _gate_norm_inputs(y, gate, weight, bias):
    if y.dim() != 4:
        raise ValueError("expected y [B,H,T,dv]")
    B, H, T, dv = _shape(y)
    dt = _dtype(y)
    _rows(y, y.shape, y, "y")
    token = (B, T, H, dv)
    if gate is not None:
        _rows(gate, token, y, "gate")
    _f32(weight, (H, dv), y, "weight")
    _f32(bias, (H, dv), y, "bias")
    return dt, B, H, T, dv, token


def _pack(*rows):
    return (ctypes.c_longlong * (3 * len(rows)))(*(s for r in rows for s in r))


def _head(t):
    return (t.stride(0), t.stride(1), t.stride(2))


def _token(t):
    return (0, 0, 0) if t is None else (t.stride(0), t.stride(2), t.stride(1))


def group_norm_gated(y: torch.Tensor, gate: Optional[torch.Tensor] = None, weight: Optional[torch.Tensor] = None,
                     bias: Optional[torch.Tensor] = None, eps: float = 1e-5, out: Optional[torch.Tensor] = None
                     ) -> torch.Tensor:
    """Per-head GroupNorm of y [B,H,T,dv] times silu(gate), heads merged (retention_group_norm_gated).

    gate, out: [B,T,H,dv], any strides with contiguous rows (a [B,T,H*dv] projection viewed by heads, or a
    slice of a fused one); without a gate the norm alone.  weight, bias: optional fp32 [H,dv].
    """
    dt, B, H, T, dv, token = _gate_norm_inputs(y, gate, weight, bias)
    if out is None:
        out = torch.empty(token, dtype=y.dtype, device=y.device) if gate is None else _like(gate)
    else:
        _rows(out, token, y, "out")
    plain = y.is_contiguous() and out.is_contiguous() and (gate is None or gate.is_contiguous())
    _call(load().retention_group_norm_gated, y.device, y.data_ptr(), _p(gate), _p(weight), _p(bias), float(eps),
          out.data_ptr(), None if plain else _pack(_head(y), _token(gate), _token(out)), B, H, T, dv, dt)
    return out


def group_norm_gated_bwd(y: torch.Tensor, gate: Optional[torch.Tensor], grad_out: torch.Tensor,
                         weight: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                         eps: float = 1e-5, param_grads: bool = True, grad_y: Optional[torch.Tensor] = None,
                         grad_gate: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None
                         ) -> Tuple[torch.Tensor, Optional[torch.Tensor], Optional[torch.Tensor],
                                    Optional[torch.Tensor]]:
    """Gradients of group_norm_gated (retention_group_norm_gated_bwd): (grad_y, grad_gate, grad_weight, grad_bias).

    With gate None the gradients of group_norm, for a token-major grad_out.  grad_weight and grad_bias (fp32)
    are None where the parameter is, or with param_grads=False.
    """
    lib = load()
    dt, B, H, T, dv, token = _gate_norm_inputs(y, gate, weight, bias)
    _rows(grad_out, token, y, "grad_out")
    gy = _like(y) if grad_y is None else _rows(grad_y, y.shape, y, "grad_y")
    if gate is None:
        gz = None
    else:
        gz = _like(gate) if grad_gate is None else _rows(grad_gate, token, y, "grad_gate")
    gw = torch.empty_like(weight) if param_grads and weight is not None else None
    gb = torch.empty_like(bias) if param_grads and bias is not None else None
    need = lib.retention_group_norm_gated_bwd_workspace_bytes(B, H, T, dv) if gw is not None or gb is not None else 0
    ws, wp, wn = _workspace(workspace, need, y)
    plain = all(t is None or t.is_contiguous() for t in (y, gate, grad_out, gy, gz))
    _call(lib.retention_group_norm_gated_bwd, y.device, y.data_ptr(), _p(gate), _p(weight), _p(bias), float(eps),
          grad_out.data_ptr(), gy.data_ptr(), _p(gz), _p(gw), _p(gb),
          None if plain else _pack(_head(y), _token(gate), _token(grad_out), _head(gy), _token(gz)), B, H, T, dv, dt,
          wp, wn)
    return gy, gz, gw, gb


# ------------------------------------------------------------- residual norm
def _row_stride(t: Optional[torch.Tensor], name: str) -> int:
    """Distance between the rows of a [...,D] tensor whose leading dimensions walk evenly."""
    if t is None:
        return 0
    if t.is_contiguous():
        return t.shape[-1]
    try:
        return t.view(-1, t.shape[-1]).stride(0)
    except RuntimeError:
        raise ValueError(f"the rows of {name} must be evenly spaced") from None


def _row_strides(**tensors):
    if all(t is None or t.is_contiguous() for t in tensors.values()):
        return None
    return (ctypes.c_longlong * len(tensors))(*(_row_stride(t, n) for n, t in tensors.items()))


def _count(t: torch.Tensor) -> Tuple[int, int]:
    if t.dim() < 1 or t.shape[-1] < 1:
        raise ValueError("expected tensors [...,D] with D >= 1")
    n, D = t.numel(), t.shape[-1]
    return (n // D, D) if n <= 0x7FFFFFFF else _sizes(n // D, D)


def residual_norm(x: torch.Tensor, f: torch.Tensor, weight: Optional[torch.Tensor] = None,
                  bias: Optional[torch.Tensor] = None, scale: Optional[torch.Tensor] = None, alpha: float = 1.0,
                  eps: float = 1e-5, rms: bool = False, r: Optional[torch.Tensor] = None,
                  n: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """r = alpha x + scale f and n = norm(r) weight + bias (retention_residual_norm): (r, n).

    x, f [...,D]: the residual stream and a block's output; weight, bias, scale: optional fp32 [D];
    LayerNorm, or RMSNorm with rms=True.
    """
    dt = _dtype(x)
    rows, D = _count(x)
    _rows(x, x.shape, x, "x")
    _rows(f, x.shape, x, "f")
    vec = (D,)
    _f32(weight, vec, x, "weight")
    _f32(bias, vec, x, "bias")
    _f32(scale, vec, x, "scale")
    r = _like(x) if r is None else _rows(r, x.shape, x, "r")
    n = _like(x) if n is None else _rows(n, x.shape, x, "n")
    _call(load().retention_residual_norm, x.device, x.data_ptr(), f.data_ptr(), _p(weight), _p(bias), _p(scale),
          float(alpha), float(eps), int(rms), r.data_ptr(), n.data_ptr(), _row_strides(x=x, f=f, r=r, n=n), rows, D, dt)
    return r, n


def residual_norm_bwd(r: torch.Tensor, grad_n: torch.Tensor, grad_r: Optional[torch.Tensor] = None,
                      weight: Optional[torch.Tensor] = None, f: Optional[torch.Tensor] = None,
                      scale: Optional[torch.Tensor] = None, alpha: float = 1.0, eps: float = 1e-5, rms: bool = False,
                      bias_grad: bool = False, param_grads: bool = True, workspace: Optional[torch.Tensor] = None):
    """Gradients of residual_norm from its stored r (retention_residual_norm_bwd):
    (grad_x, grad_f, grad_weight, grad_bias, grad_scale).

    grad_r: what reaches r from later in the stream (None: nothing).  f is needed for grad_scale only.
    grad_weight and grad_scale are None where the parameter is (or with param_grads=False), grad_bias without
    bias_grad.  With alpha = 1 and no scale the gradients of x and f are equal and grad_f is grad_x itself.
    """
    lib = load()
    dt = _dtype(r)
    rows, D = _count(r)
    _rows(r, r.shape, r, "r")
    _rows(grad_n, r.shape, r, "grad_n")
    for t, name in ((grad_r, "grad_r"), (f, "f")):
        if t is not None:
            _rows(t, r.shape, r, name)
    vec = (D,)
    _f32(weight, vec, r, "weight")
    _f32(scale, vec, r, "scale")
    want_scale = param_grads and scale is not None
    if want_scale and f is None:
        raise ValueError("f is required for the gradient of scale")
    gx = _like(r)
    same = alpha == 1.0 and scale is None
    gf = None if same else torch.empty_like(gx)
    gw = torch.empty_like(weight) if param_grads and weight is not None else None
    gb = torch.empty(D, dtype=torch.float32, device=r.device) if param_grads and bias_grad else None
    gs = torch.empty_like(scale) if want_scale else None
    need = 0
    if gw is not None or gb is not None or gs is not None:
        need = lib.retention_residual_norm_bwd_workspace_bytes(rows, D)
    ws, wp, wn = _workspace(workspace, need, r)
    ff = f if want_scale else None
    _call(lib.retention_residual_norm_bwd, r.device, r.data_ptr(), grad_n.data_ptr(), _p(grad_r), _p(ff), _p(weight),
          _p(scale), float(alpha), float(eps), int(rms), gx.data_ptr(), _p(gf), _p(gw), _p(gb), _p(gs),
          _row_strides(r=r, grad_n=grad_n, grad_r=grad_r, f=ff, grad_x=gx, grad_f=gf), rows, D, dt, wp, wn)
    return gx, (gx if same else gf), gw, gb, gs

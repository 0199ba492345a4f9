"""libretention: multi-scale retention on AMD Instinct MI355X (gfx950).

The compute lives in hand-written HIP kernels behind a C ABI
(include/libretention.h); this package is the thin Python binding:

    chunkwise_fwd(q, k, v, gamma, C, state_in=None, state_out=True) -> (y, state_out)
    chunkwise_fwd_noalloc(q, k, v, gamma, C, state_in=None, state_out=None, y=None) -> y
        (the same with no allocation inside the call: static device scratch)
    chunkwise_bwd(q, k, v, gamma, C, grad_y, state_in=None, grad_state_out=None)
        -> (grad_q, grad_k, grad_v, grad_state_in)
    parallel_fwd(q, k, v, gamma, state_in=None) -> y
    recurrent_step(q, k, v, gamma, state) -> y          (state updated in place)
    group_norm(y, weight=None, bias=None, eps=1e-5) -> out   (per-head GroupNorm of y)
    chunkwise_fwd_group_norm(q, k, v, gamma, C, weight=None, bias=None, eps=1e-5, ...)
        -> (y, state_out)     (the forward with the GroupNorm fused into its stores)
    fused_group_norm_failed(workspace, B, H, T, dk, dv, C, dtype) -> bool
        (whether a wait of that fused call gave up; its error word)

Around retention in a block (strided tensors: any layout with contiguous rows):

    gated_scan_fwd(x, f, rate, state_in=None, state_out=True, normalize=False, checkpoints=None)
        -> (y, state_out[, checkpoints])   (h_t = sigmoid(f_t)^rate h_(t-1) + u_t)
    gated_scan_bwd(x, f, rate, grad_y, state_in=None, grad_state_out=None, checkpoints=None, normalize=False)
        -> (grad_x, grad_f, grad_state_in)
    gated_scan_step(x, f, rate, state, normalize=False) -> y      (state updated in place)
    group_norm_gated(y, gate=None, weight=None, bias=None, eps=1e-5) -> out
        (per-head GroupNorm of y [B,H,T,dv] times silu(gate), gate and out [B,T,H,dv])
    group_norm_gated_bwd(y, gate, grad_out, weight=None, bias=None, eps=1e-5)
        -> (grad_y, grad_gate, grad_weight, grad_bias)      (gate=None: of group_norm)
    residual_norm(x, f, weight=None, bias=None, scale=None, alpha=1.0, eps=1e-5, rms=False) -> (r, n)
        (r = alpha x + scale f, n = LayerNorm or RMSNorm of r)
    residual_norm_bwd(r, grad_n, grad_r=None, weight=None, f=None, scale=None, ...)
        -> (grad_x, grad_f, grad_weight, grad_bias, grad_scale)

Softmax attention beside retention in a hybrid stack (one map, or the difference of two with lam):

    attention_fwd(q, k, v, lam=None, causal=True, scale=None, offset=None, lens=None, keep=False)
        -> o  or  (o, kept)     (query heads may share key heads; kept is for the backward)
    attention_bwd(q, k, v, o, grad_o, kept, lam=None, causal=True, scale=None, offset=None, lens=None)
        -> (grad_q, grad_k, grad_v, grad_lam)
    attention_step(q, k, v, k_cache, v_cache, table, lens, lam=None, scale=None) -> o
        (one new token of every sequence, in place on a paged cache)
    cache_append(k, v, k_cache, v_cache, table, start, counts=None)   (a prompt's keys and values into the cache)

Build the library with ``python -m retnet_retention_chunkwise_amd.build``.
"""
from ._attention import (  # noqa: F401
    attention_bwd,
    attention_fwd,
    attention_step,
    cache_append,
)
from ._block import (  # noqa: F401
    gated_scan_bwd,
    gated_scan_checkpoint_shape,
    gated_scan_fwd,
    gated_scan_step,
    group_norm_gated,
    group_norm_gated_bwd,
    residual_norm,
    residual_norm_bwd,
)
from ._lib import (  # noqa: F401
    LIB_PATH,
    MAX_CHUNK,
    MAX_DK,
    MAX_DV,
    RetentionError,
    chunkwise_bwd,
    chunkwise_fwd,
    chunkwise_fwd_group_norm,
    chunkwise_fwd_noalloc,
    chunkwise_workspace_bytes,
    fused_group_norm_failed,
    group_norm,
    last_error,
    load,
    parallel_fwd,
    recurrent_step,
    testing_gn_wait,
    version,
)

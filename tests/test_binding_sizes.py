"""Sizes of 2^31 and more do not fit the C ABI's ints: every call of the binding refuses them, where ctypes by itself
would pass their low 32 bits and so work on a small part of the tensors (no GPU: the tensors are one element
expanded, and sizes are looked at before devices)."""
import pytest
import torch

import retnet_retention_chunkwise_amd as ret
from retnet_retention_chunkwise_amd import _lib

BIG = 2 ** 32 + 2


def t(*shape, dtype=torch.float32):
    return torch.zeros(1, dtype=dtype).expand(*shape)


@pytest.mark.parametrize("shape", [(BIG, 2, 3, 4), (1, BIG, 3, 4), (1, 2, BIG, 4), (1, 2, 3, BIG), (BIG, 2, 0, 4),
                                   (1, 2, 2 ** 31, 1)])
def test_tensor_dimensions(shape):
    B, H, T, d = shape
    x, step, rate = t(*shape), t(B, H, d), [1.0, 0.5]
    token = t(B, T, H, d)
    calls = [lambda: ret.gated_scan_fwd(x, x, rate), lambda: ret.gated_scan_bwd(x, x, rate, x),
             lambda: ret.group_norm_gated(x, token), lambda: ret.group_norm_gated_bwd(x, token, token),
             lambda: ret.parallel_fwd(x, x, x, rate), lambda: ret.chunkwise_fwd(x, x, x, rate, 64),
             lambda: ret.chunkwise_fwd(x[..., :2], x[..., :2], x, rate, 64),
             lambda: ret.chunkwise_fwd_group_norm(x, x, x, rate, 64), lambda: ret.chunkwise_bwd(x, x, x, rate, 64, x),
             lambda: ret.chunkwise_fwd_noalloc(x, x, x, rate, 64)]
    if max(B, H, d) > 2 ** 31:
        calls += [lambda: ret.gated_scan_step(step, step, rate, step),
                  lambda: ret.recurrent_step(step, step, step, rate, step)]
    for call in calls:
        with pytest.raises(ValueError, match="below 2\\^31"):
            call()


@pytest.mark.parametrize("shape", [(2 ** 32 + 8, 1), (2 ** 16, 2 ** 16, 4), (1, 2 ** 31), (2 ** 31, 1)])
def test_rows_of_a_residual_stream(shape):
    x = t(*shape)
    for call in (lambda: ret.residual_norm(x, x), lambda: ret.residual_norm_bwd(x, x)):
        with pytest.raises(ValueError, match="below 2\\^31"):
            call()


def test_sizes_given_as_numbers():
    for bad in ((BIG, 3, 1, 64), (1, BIG, 1, 64), (1, 3, BIG, 64), (1, 3, 1, BIG), (1, 1, -BIG, 1)):
        with pytest.raises(ValueError, match="below 2\\^31"):
            ret.gated_scan_checkpoint_shape(*bad)
    for i in range(6):
        args = [1, 2, 256, 64, 64, 64]
        args[i] = BIG
        with pytest.raises(ValueError, match="below 2\\^31"):
            ret.chunkwise_workspace_bytes(*args, torch.bfloat16)
        with pytest.raises(ValueError, match="below 2\\^31"):
            ret.fused_group_norm_failed(None, *args, torch.bfloat16)
    x = t(1, 2, 8, 4)
    for call in (ret.chunkwise_fwd, ret.chunkwise_fwd_group_norm, ret.chunkwise_fwd_noalloc):
        with pytest.raises(ValueError, match="below 2\\^31"):
            call(x, x, x, [1.0, 0.5], 2 ** 32 + 64)
    # what fits goes on to the library, which names what it refuses
    assert ret.gated_scan_checkpoint_shape(2, 3, 300, 64) == (2, 3, 3, 64)
    with pytest.raises(ret.RetentionError, match="B=-1"):
        ret.gated_scan_checkpoint_shape(-1, 3, 300, 64)
    assert _lib._sizes(2 ** 31 - 1, 0) == (2 ** 31 - 1, 0)

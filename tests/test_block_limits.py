"""Sizes at the limits of the block operators' calls: what a launch cannot take is refused with its name before
anything is enqueued (no GPU: made-up addresses, never dereferenced)."""
import ctypes

import pytest

from retnet_retention_chunkwise_amd import _lib

INVALID, UNSUPPORTED = _lib.RET_ERR_INVALID_ARG, _lib.RET_ERR_UNSUPPORTED
BAD = ctypes.c_size_t(-1).value


def at(n):
    return ctypes.c_void_p(n << 36)


@pytest.mark.parametrize("with_checkpoints", [True, False])
@pytest.mark.parametrize("B,H,d", [((1 << 21) + 1, 1, 1), (1 << 17, 128, 1), (1 << 15, 128, 16)])
def test_backward_of_one_token_refuses_more_runs_than_a_launch_takes(B, H, d, with_checkpoints):
    """2^24 runs of 512 threads would be 2^33 threads; a grid has fewer than 2^32."""
    lib = _lib.load()
    rate = (ctypes.c_float * H)(*[1.0] * H)
    ck = at(7) if with_checkpoints else None
    st = lib.retention_gated_scan_bwd(at(1), at(2), rate, None, ck, at(3), None, at(4), at(5), None, None, B, H, 1, d, 0,
                                      0, at(9), 1 << 36, None)
    assert st == UNSUPPORTED and "2^21" in _lib.last_error(), _lib.last_error()
    assert lib.retention_gated_scan_bwd_workspace_bytes(B, H, 1, d, 0, int(with_checkpoints)) == BAD
    assert "2^21" in _lib.last_error()
    # the forward of one token goes by the element
    assert lib.retention_gated_scan_workspace_bytes(B, H, 1, d, 0) == 0


@pytest.mark.parametrize("B,H,d,most", [
    (1 << 12, 32, 512, 1 << 20), (1 << 13, 32, 512, 1 << 21), (1 << 14, 64, 65, 1 << 21), (1 << 16, 32, 64, 1 << 21),
    (1 << 16, 16, 48, 1 << 20), (1 << 15, 64, 32, 1 << 21), (1 << 16, 32, 16, 1 << 21), (1 << 21, 1, 3, 1 << 21)])
def test_tiles_are_counted_as_wide_as_the_kernels_take_them(B, H, d, most):
    """Rows of more than 32 channels are walked 64 channels at a time, of more than 16 32: at most 2^21 tiles."""
    lib = _lib.load()
    w = 64 if d > 32 else 32 if d > 16 else 16
    assert B * H * -(-d // w) == most
    for size in (lambda b: lib.retention_gated_scan_workspace_bytes(b, H, 2, d, 1),
                 lambda b: lib.retention_gated_scan_bwd_workspace_bytes(b, H, 2, d, 1, 1)):
        assert size(B) == 0  # so many runs are walked, without a workspace
        if most == 1 << 21:
            assert size(B + 1) == BAD and "2^21" in _lib.last_error()

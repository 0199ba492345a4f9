"""The range of the attention calls' scale (no GPU: every call below fails validation, or has no rows, before any HIP call)."""
import pytest

from retnet_retention_chunkwise_amd import _lib
from test_attention_abi import INVALID, UNSUPPORTED, at, bwd, fwd, lib, step  # noqa: F401

OUT = [2.0 ** -101, 1.6e-38, 1.2e-38, 1e-45, 2.0 ** 101, 2.4e38, 3.4e38]


@pytest.mark.parametrize("call", [fwd, bwd, step])
@pytest.mark.parametrize("scale", OUT)
def test_scales_out_of_range_are_refused(lib, call, scale):  # noqa: F811
    """Scales whose exponent arguments, or the slack of the running maximum, would leave fp32."""
    assert call(lib, scale=scale) == UNSUPPORTED
    assert "scale" in _lib.last_error() and "2^100" in _lib.last_error(), _lib.last_error()


@pytest.mark.parametrize("scale", [0.0, -2.0 ** -101, float("inf"), float("nan")])
def test_no_scales_are_invalid(lib, scale):  # noqa: F811
    for call in (fwd, bwd, step):
        assert call(lib, scale=scale) == INVALID and "scale" in _lib.last_error()


def test_the_ends_of_the_range_are_taken(lib):  # noqa: F811
    for scale in (2.0 ** -100, 2.0 ** 100):
        assert fwd(lib, T=0, scale=scale) == 0
        # past the scale: the next check's refusal
        assert bwd(lib, lse=None, scale=scale) == INVALID and "lse" in _lib.last_error()
        assert step(lib, lens=None, scale=scale) == INVALID and "lens" in _lib.last_error()

"""Pins of the block operators' oracle (CPU): hand values, library routines and
central differences, none of which re-types the oracle."""
import math

import pytest
import torch

import oracle

F64 = torch.float64


def _rand(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=F64)


def differences(fn, t, eps=1e-6):
    """Central differences of the scalar fn() with respect to every entry of t."""
    g = torch.empty_like(t)
    flat, gf = t.view(-1), g.view(-1)
    for i in range(flat.numel()):
        keep = flat[i].item()
        flat[i] = keep + eps
        up = fn()
        flat[i] = keep - eps
        down = fn()
        flat[i] = keep
        gf[i] = (up - down) / (2 * eps)
    return g


# ------------------------------------------------------------- gated scan
def test_scan_hand_values():
    # f = 0: a = 1/2 at rate 1 and 1/4 at rate 2; x = 8, 4, 4
    x = torch.tensor([8.0, 4.0, 4.0], dtype=F64).view(1, 1, 3, 1).repeat(1, 2, 1, 1)
    f = torch.zeros_like(x)
    h, last = oracle.gated_scan(x, f, [1.0, 2.0])
    assert torch.allclose(h[0, 0, :, 0], torch.tensor([8.0, 8.0, 8.0], dtype=F64))
    assert torch.allclose(h[0, 1, :, 0], torch.tensor([8.0, 6.0, 5.5], dtype=F64))
    assert torch.equal(last, h[:, :, -1])
    h, _ = oracle.gated_scan(x, f, [1.0, 2.0], torch.full((1, 2, 1), 16.0), normalize=True)
    assert torch.allclose(h[0, 0, :, 0], torch.tensor([12.0, 8.0, 6.0], dtype=F64))
    assert torch.allclose(h[0, 1, :, 0], torch.tensor([10.0, 5.5, 4.375], dtype=F64))


def test_scan_gate_limits():
    """f = -inf forgets everything before, f = +inf keeps all of it."""
    x, s = _rand(1, 1, 4, 3, seed=1), _rand(1, 1, 3, seed=2)
    f = torch.full_like(x, math.inf)
    f[:, :, 2] = -math.inf
    h, _ = oracle.gated_scan(x, f, [0.5], s)
    assert torch.allclose(h[:, :, 1], s + x[:, :, 0] + x[:, :, 1])
    assert torch.equal(h[:, :, 2], x[:, :, 2])
    h, _ = oracle.gated_scan(x, f, [0.5], s, normalize=True)
    assert torch.equal(h[:, :, 1], s) and torch.equal(h[:, :, 2], x[:, :, 2]) and torch.equal(h[:, :, 3], x[:, :, 2])
    gx, gf, gs = oracle.gated_scan_backward(x, f, [0.5], torch.ones_like(x), s)
    assert torch.equal(gf, torch.zeros_like(gf)) and torch.equal(gs, torch.full_like(gs, 2.0))


def test_scan_is_retention_with_one_key_channel():
    """A gate that is the same for every token is retention with d_k = 1, q = k = 1."""
    x = _rand(2, 3, 17, 5, seed=3)
    rate = [1.0, 0.5, 0.25]
    h, last = oracle.gated_scan(x, torch.full_like(x, 1.5), rate)
    gamma = torch.sigmoid(torch.tensor(1.5, dtype=F64)) ** torch.tensor(rate, dtype=F64)
    one = torch.ones(2, 3, 17, 1, dtype=F64)
    y, state = oracle.recurrent(one, one, x, gamma)
    assert torch.allclose(h, y, atol=1e-12) and torch.allclose(last, state[:, :, 0], atol=1e-12)


@pytest.mark.parametrize("normalize", [False, True])
def test_scan_gradients_match_differences(normalize):
    B, H, T, d = 1, 2, 5, 3
    x, f, s = _rand(B, H, T, d, seed=4), _rand(B, H, T, d, seed=5) + 1, _rand(B, H, d, seed=6)
    dy, ds = _rand(B, H, T, d, seed=7), _rand(B, H, d, seed=8)
    rate = [1.0, 0.25]

    def loss():
        h, last = oracle.gated_scan(x, f, rate, s, normalize)
        return float((h * dy).sum() + (last * ds).sum())

    got = oracle.gated_scan_backward(x, f, rate, dy, s, ds, normalize)
    for g, t in zip(got, (x, f, s)):
        assert torch.allclose(g, differences(loss, t), atol=1e-7), (normalize, (g - differences(loss, t)).abs().max())


def test_scan_planted_slips_fail():
    """The differences tell a wrong gradient from the right one."""
    x, f, dy = _rand(1, 1, 4, 2, seed=9), _rand(1, 1, 4, 2, seed=10), _rand(1, 1, 4, 2, seed=11)
    gx, gf, _ = oracle.gated_scan_backward(x, f, [0.5], dy, normalize=True)
    loss = lambda: float((oracle.gated_scan(x, f, [0.5], normalize=True)[0] * dy).sum())  # noqa: E731
    want = differences(loss, f)
    plain = oracle.gated_scan_backward(x, f, [0.5], dy, normalize=False)[1]
    no_rate = oracle.gated_scan_backward(x, f, [1.0], dy, normalize=True)[1]
    for slip in (plain, no_rate, -gf, gf.flip(2)):
        assert not torch.allclose(slip, want, atol=1e-4)


# ----------------------------------------------------------- gated GroupNorm
def test_gate_norm_against_library_routines():
    B, H, T, dv = 2, 3, 4, 6
    y, z, w, b = _rand(B, H, T, dv, seed=20), _rand(B, T, H, dv, seed=21), _rand(H, dv, seed=22), _rand(H, dv, seed=23)
    merged = y.transpose(1, 2).reshape(B * T, H * dv)
    n = torch.nn.functional.group_norm(merged, H, w.reshape(-1), b.reshape(-1), 1e-3).view(B, T, H, dv)
    assert torch.allclose(oracle.group_norm_gated(y, None, w, b, 1e-3), n, atol=1e-12)
    assert torch.allclose(oracle.group_norm_gated(y, z, w, b, 1e-3), n * torch.nn.functional.silu(z), atol=1e-12)
    # without a gate and transposed back it is the plain per-head norm
    assert torch.allclose(oracle.group_norm_gated(y, None, w, b, 1e-3).transpose(1, 2), oracle.group_norm(y, w, b, 1e-3))


def test_gate_norm_hand_values():
    # y = 1, 3: mu = 2, variance 1, xh = -1, 1; silu(0) = 0, silu(ln 3) = 0.75 ln 3
    y = torch.tensor([1.0, 3.0], dtype=F64).view(1, 1, 1, 2)
    z = torch.tensor([0.0, math.log(3.0)], dtype=F64).view(1, 1, 1, 2)
    got = oracle.group_norm_gated(y, z, torch.tensor([[2.0, 2.0]]), torch.tensor([[1.0, 1.0]]), 0.0)
    assert torch.allclose(got.view(-1), torch.tensor([0.0, 3.0 * 0.75 * math.log(3.0)], dtype=F64))


@pytest.mark.parametrize("gated", [False, True])
def test_gate_norm_gradients_match_differences(gated):
    B, H, T, dv = 2, 2, 2, 5
    y, z = _rand(B, H, T, dv, seed=24), _rand(B, T, H, dv, seed=25) if gated else None
    w, b, do = _rand(H, dv, seed=26), _rand(H, dv, seed=27), _rand(B, T, H, dv, seed=28)
    loss = lambda: float((oracle.group_norm_gated(y, z, w, b, 1e-2) * do).sum())  # noqa: E731
    gy, gz, gw, gb = oracle.group_norm_gated_backward(y, z, do, w, b, 1e-2)
    for g, t in ((gy, y), (gz, z), (gw, w), (gb, b)):
        if t is not None:
            assert torch.allclose(g, differences(loss, t), atol=1e-7)


# ------------------------------------------------------------- residual norm
def test_stream_norm_against_library_routines():
    r, w, b = _rand(7, 9, seed=30), _rand(9, seed=31), _rand(9, seed=32)
    assert torch.allclose(oracle.stream_norm(r, w, b, 1e-3), torch.nn.functional.layer_norm(r, (9,), w, b, 1e-3))
    assert torch.allclose(oracle.stream_norm(r, w, None, 1e-3, True), torch.nn.functional.rms_norm(r, (9,), w, 1e-3))
    x = torch.tensor([2.0, -4.0], dtype=F64)
    assert torch.equal(oracle.residual(x, x, torch.tensor([1.0, 0.5]), 3.0), torch.tensor([8.0, -14.0], dtype=F64))


@pytest.mark.parametrize("rms", [False, True])
def test_residual_norm_gradients_match_differences(rms):
    R, D, alpha = 3, 5, 1.5
    x, f, w, b, s = _rand(R, D, seed=33), _rand(R, D, seed=34), _rand(D, seed=35), _rand(D, seed=36), _rand(D, seed=37)
    dn, dr = _rand(R, D, seed=38), _rand(R, D, seed=39)

    def loss():
        r = oracle.residual(x, f, s, alpha)
        return float((oracle.stream_norm(r, w, b, 1e-2, rms) * dn).sum() + (r * dr).sum())

    got = oracle.residual_norm_backward(oracle.residual(x, f, s, alpha), dn, dr, w, f, s, alpha, 1e-2, rms)
    for g, t in zip(got, (x, f, w, b, s)):
        assert torch.allclose(g, differences(loss, t), atol=1e-7)
    slip = oracle.residual_norm_backward(oracle.residual(x, f, s, alpha), dn, dr, w, f, s, alpha, 1e-2, not rms)
    assert not torch.allclose(slip[0], differences(loss, x), atol=1e-3)

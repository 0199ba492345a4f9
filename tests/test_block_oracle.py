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

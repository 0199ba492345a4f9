"""Pins of the attention oracle (CPU): hand values, library routines and central
differences, none of which re-types the oracle."""
import math

import pytest
import torch

import oracle

F64 = torch.float64


def _rand(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=F64)


def test_hand_values():
    # keys 0 and ln 3 at scale 1 and q = 1: weights 1/4 and 3/4
    q = torch.ones(1, 1, 2, 1, dtype=F64)
    k = torch.tensor([0.0, math.log(3)], dtype=F64).view(1, 1, 2, 1)
    v = torch.tensor([4.0, 8.0], dtype=F64).view(1, 1, 2, 1)
    o, lse, second = oracle.attention(q, k, v, causal=True, scale=1.0)
    assert torch.allclose(o.flatten(), torch.tensor([4.0, 7.0], dtype=F64)) and second is None
    assert torch.allclose(lse.flatten(), torch.tensor([0.0, math.log(4)], dtype=F64))
    # a second map with equal scores: its mean is 6
    q2, k2 = torch.cat([q, q], -1), torch.cat([k, 0 * k], -1)
    o, lse, second = oracle.attention(q2, k2, v, torch.tensor([0.5]), causal=False, scale=1.0)
    assert torch.allclose(second.flatten(), torch.full((2,), 6.0, dtype=F64))
    assert torch.allclose(o.flatten(), torch.full((2,), 7.0 - 0.5 * 6.0, dtype=F64))
    assert torch.allclose(lse[0, 0, 1], torch.full((2,), math.log(2), dtype=F64))


@pytest.mark.parametrize("causal", [True, False])
def test_ordinary_is_the_library_routine(causal):
    q, k, v = _rand(2, 6, 9, 8, seed=1), _rand(2, 2, 9, 8, seed=2), _rand(2, 2, 9, 5, seed=3)
    want = torch.nn.functional.scaled_dot_product_attention(q, k.repeat_interleave(3, 1), v.repeat_interleave(3, 1),
                                                            is_causal=causal)
    assert torch.allclose(oracle.attention(q, k, v, causal=causal)[0], want)


def test_differential_is_a_difference_of_ordinary_ones():
    q, k, v, lam = _rand(1, 4, 7, 6, seed=1), _rand(1, 2, 7, 6, seed=2), _rand(1, 2, 7, 5, seed=3), _rand(4, seed=4)
    o, _, second = oracle.attention(q, k, v, lam)
    a = oracle.attention(q[..., :3], k[..., :3], v)[0]
    b = oracle.attention(q[..., 3:], k[..., 3:], v)[0]
    assert torch.allclose(second, b) and torch.allclose(o, a - lam.view(1, 4, 1, 1) * b)


def test_rows_without_keys_and_padding():
    q, k, v = _rand(2, 2, 5, 4, seed=1), _rand(2, 2, 3, 4, seed=2), _rand(2, 2, 3, 4, seed=3)
    o, lse, _ = oracle.attention(q, k, v)  # offset -2: the first two rows see nothing
    assert torch.equal(o[:, :, :2], torch.zeros(2, 2, 2, 4, dtype=F64)) and torch.isneginf(lse[..., :2]).all()
    assert torch.allclose(o[:, :, 2], v[:, :, 0])
    k[0, :, 2:], v[0, :, 2:] = math.nan, math.inf
    o, _, _ = oracle.attention(q, k, v, lens=torch.tensor([2, 0]), causal=False)
    want = oracle.attention(q[:1], k[:1, :, :2], v[:1, :, :2], causal=False)[0]
    assert torch.allclose(o[:1], want) and torch.equal(o[1], torch.zeros_like(o[1]))


@pytest.mark.parametrize("two,causal,lens", [(True, True, None), (True, False, [4, 0]), (False, True, [3, 5])])
def test_gradients_by_differences(two, causal, lens):
    q, k, v = _rand(2, 2, 4, 4, seed=1), _rand(2, 1, 5, 4, seed=2), _rand(2, 1, 5, 3, seed=3)
    lam = _rand(2, seed=4) if two else None
    do = _rand(2, 2, 4, 3, seed=5)
    lens = None if lens is None else torch.tensor(lens)
    loss = lambda: float((do * oracle.attention(q, k, v, lam, causal, 0.7, lens=lens)[0]).sum())  # noqa: E731
    grads = oracle.attention_backward(q, k, v, do, lam, causal, 0.7, lens=lens)
    for t, g in zip((q, k, v, lam), grads):
        if t is None:
            assert g is None
            continue
        flat, gf = t.view(-1), g.reshape(-1)
        for i in range(flat.numel()):
            keep = flat[i].item()
            flat[i] = keep + 1e-6
            up = loss()
            flat[i] = keep - 1e-6
            down = loss()
            flat[i] = keep
            assert abs((up - down) / 2e-6 - gf[i].item()) < 1e-7


def test_step_is_the_last_row():
    """A step over pages is the last row of a causal call over the same tokens in order."""
    B, H, Hk, n, dk, dv, page = 2, 4, 2, 11, 4, 3, 4
    q, k, v = _rand(B, H, n, dk, seed=1), _rand(B, Hk, n, dk, seed=2), _rand(B, Hk, n, dv, seed=3)
    table = torch.tensor([[5, 0, 3], [1, 6, 2]])
    kc, vc = torch.full((7, Hk, page, dk), math.nan, dtype=F64), torch.full((7, Hk, page, dv), math.nan, dtype=F64)
    lam = _rand(H, seed=4)
    kc, vc = oracle.cache_append(k, v, kc, vc, table, torch.tensor([0, 0]), torch.tensor([10, 10]))
    assert torch.equal(kc[3, :, 1], k[0, :, 9]) and torch.isnan(kc[3, :, 2]).all() and torch.isnan(kc[4]).all()
    o, kc, vc = oracle.attention_step(q[:, :, 10], k[:, :, 10], v[:, :, 10], kc, vc, table, torch.tensor([10, 10]), lam)
    assert torch.allclose(o, oracle.attention(q, k, v, lam)[0][:, :, 10])
    assert torch.equal(vc[2, :, 2], v[1, :, 10])
    # a page that is not there hides its tokens; an idle sequence is zero and stores nothing
    gone = table.clone()
    gone[0, 0] = 7
    o, kc2, _ = oracle.attention_step(q[:, :, 10], k[:, :, 10], v[:, :, 10], kc, vc, gone, torch.tensor([10, -1]), lam)
    want = oracle.attention(q[:1, :, 10:], k[:1, :, 4:], v[:1, :, 4:], lam)[0][0, :, 0]
    assert torch.allclose(o[0], want) and torch.equal(o[1], torch.zeros_like(o[1]))

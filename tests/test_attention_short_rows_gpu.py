"""bf16 gradients of rows that see at most 32 keys, beside rows that see more: each within the bounds of a mean
that comes from the row's weights, whatever the other rows of its tile see."""
import pytest
import torch

import oracle
import retnet_retention_chunkwise_amd as ret
from attention_bounds import bounds, close
from helpers import say

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16 = torch.bfloat16


def rnd(g, *shape, scale=1.0):
    return (torch.randn(shape, generator=g) * scale).to(BF16)


def seen(T, S, offset, lens):
    """[B,T]: keys that each row sees."""
    n = torch.tensor(lens)[:, None]
    return torch.minimum((torch.arange(T)[None] + offset + 1).clamp_min(0), n)


@pytest.mark.parametrize("two", [True, False])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (256, 40), (200, 256), (90, 33), (256, 256)])
@pytest.mark.parametrize("T,S,offset,lens", [
    (64, 65, 1, None), (64, 68, 4, None), (96, 105, 9, None), (70, 101, 31, None), (96, 76, -20, None), (130, 120, -10, None),
    (64, 64, 3, [64, 20]), (20, 900, 1, None), (40, 700, 17, [700, 33]),  # the last ones with the keys split
])
def test_gradients(T, S, offset, lens, dk, dv, two):
    B, H, Hk = 2, 4, 2
    say(f"short rows T{T} S{S} offset {offset} lens {lens} dk{dk} dv{dv} maps={1 + two}")
    g = torch.Generator().manual_seed(T + S + dk + dv)
    q, k, v, do = rnd(g, B, H, T, dk, scale=1.5), rnd(g, B, Hk, S, dk), rnd(g, B, Hk, S, dv), rnd(g, B, H, T, dv)
    lam = torch.randn(H, generator=g) * 0.3 + 0.6 if two else None
    n = seen(T, S, offset, [S] * B if lens is None else lens)
    assert (n <= 32).any()
    # only short rows have a gradient: it is theirs alone that reaches the keys
    do = torch.where((n <= 32)[:, None, :, None], do, torch.zeros_like(do))
    m = dict(causal=True, offset=offset, lens=None if lens is None else torch.tensor(lens, dtype=torch.int32))
    dm = dict(m, lens=None if lens is None else m["lens"].to(DEV))
    a = [None if t is None else t.to(DEV) for t in (q, k, v, lam, do)]
    o, kept = ret.attention_fwd(*a[:4], keep=True, **dm)
    grads = ret.attention_bwd(*a[:3], o, a[4], kept, a[3], **dm)
    want = oracle.attention_backward(q, k, v, do, lam, **m)
    lim = bounds(q, k, v, lam, grad_o=do, few=True, **m)
    for name, x, w in zip(("gq", "gk", "gv", "gl"), grads, want):
        if w is not None:
            close(name, x, w, lim[name])
    assert (grads[0].cpu()[(n > 32)[:, None].expand(B, H, T)] == 0).all()
    again = ret.attention_bwd(*a[:3], o, a[4], kept, a[3], **dm)
    assert all(x is y or torch.equal(x, y) for x, y in zip(grads, again))


def test_one_row_of_two_keys():
    """A row of two keys at the head of a tile of long ones: the gradient's own size, not that of what cancels in it."""
    T, S, d = 64, 65, 64
    g = torch.Generator().manual_seed(3)
    worst = 0.0
    for _ in range(20):
        q, k, v, do = rnd(g, 1, 1, T, d), rnd(g, 1, 1, S, d), rnd(g, 1, 1, S, d), rnd(g, 1, 1, T, d)
        a = [t.to(DEV) for t in (q, k, v)]
        o, kept = ret.attention_fwd(*a, keep=True)
        got = ret.attention_bwd(*a, o, do.to(DEV), kept)[0].cpu().double()[0, 0, 0]
        want = oracle.attention_backward(q, k, v, do)[0][0, 0, 0]
        worst = max(worst, float((got - want).norm() / want.norm()))
    say(f"rows of two keys: worst relative error {worst:.4f}")
    # dS of either key and the output rounded by 2^-8 at most, the fp32 mean by far less
    assert worst <= 2 * 2.0 ** -8 + 2.0 ** -12

"""Keys and values that a causal mask hides from every row, as the unwritten end of a longer buffer has them: whatever
they hold, outputs and gradients are those of any other filling, and their own gradients are zero."""
import pytest
import torch

import retnet_retention_chunkwise_amd as ret
from helpers import say

pytestmark = pytest.mark.gpu

DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


@pytest.mark.parametrize("two", [True, False])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (256, 256), (192, 96), (50, 131)])
@pytest.mark.parametrize("T,S,offset,lens", [
    (70, 200, 50, None),       # the last row's limit inside a tile, and whole tiles behind it
    (1, 300, 9, None),
    (33, 64, -2, [40, 64]),    # rows that see nothing in front
    (40, 2000, 700, None),     # the keys are split
    (300, 333, 0, [333, 310]),  # the rows are shared out
])
def test_hidden_keys_are_not_used(T, S, offset, lens, dk, dv, dtype, two):
    B, H, Hk = 2, 4, 2
    say(f"hidden keys T{T} S{S} offset {offset} lens {lens} dk{dk} dv{dv} {dtype} maps={1 + two}")
    g = torch.Generator().manual_seed(T + S + dk)
    q, k, v, do = (torch.randn(s, generator=g).to(dtype).to(DEV) for s in ((B, H, T, dk), (B, Hk, S, dk), (B, Hk, S, dv), (B, H, T, dv)))
    lam = torch.rand(H, generator=g).to(DEV) if two else None
    m = dict(causal=True, offset=offset, lens=None if lens is None else torch.tensor(lens, dtype=torch.int32, device=DEV))
    last = T + offset  # keys that the last row sees

    def both(kk, vv):
        o, kept = ret.attention_fwd(q, kk, vv, lam, keep=True, **m)
        return (o, *kept, *ret.attention_bwd(q, kk, vv, o, do, kept, lam, **m))

    k[:, :, last:], v[:, :, last:] = 0, 0
    want = both(k, v)
    assert all(x is None or torch.isfinite(x[x != -torch.inf]).all() for x in want)
    for a, b in ((float("nan"), 0), (0, float("nan")), (float("inf"), -float("inf")), (1e38, 1e38)):
        kk, vv = k.clone(), v.clone()
        kk[:, :, last:], vv[:, :, last:] = a, b
        got = both(kk, vv)
        assert all(x is y or torch.equal(x, y) for x, y in zip(got, want)), (a, b)
        assert (got[-3][:, :, last:] == 0).all() and (got[-2][:, :, last:] == 0).all()

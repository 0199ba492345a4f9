"""Attention at the ends of its range of scales: the bits of the same scores at an ordinary scale."""
import pytest
import torch

import retnet_retention_chunkwise_amd as ret
from helpers import say

pytestmark = pytest.mark.gpu

DEV = "cuda"
F32, BF16, I32 = torch.float32, torch.bfloat16, torch.int32
USUAL = 2.0 ** -3
# scale, and the powers of two that q and k are multiplied by to have the scores of USUAL
ENDS = [(2.0 ** -100, 2.0 ** 48, 2.0 ** 49), (2.0 ** 100, 2.0 ** -52, 2.0 ** -51)]


def ints(g, *shape, dtype):
    """Whole numbers -2..2: every product and sum of scores is exact, at any power of two."""
    return torch.randint(-2, 3, shape, generator=g).to(dtype).to(DEV)


@pytest.mark.parametrize("scale,a,b", ENDS)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,H,Hk,T,S,dk,dv", [(2, 4, 2, 100, 100, 64, 48), (1, 2, 1, 9, 1500, 128, 128), (1, 2, 2, 40, 40, 30, 201)])
def test_whole_sequences(B, H, Hk, T, S, dk, dv, dtype, scale, a, b):
    assert USUAL == scale * a * b
    g = torch.Generator().manual_seed(T + S)
    q, k = ints(g, B, H, T, dk, dtype=dtype), ints(g, B, Hk, S, dk, dtype=dtype)
    v, do = (torch.randn(s, generator=g).to(dtype).to(DEV) for s in ((B, Hk, S, dv), (B, H, T, dv)))
    for lam in (None, torch.rand(H, generator=g).to(DEV)):
        say(f"scale {scale:.3g} T{T} S{S} {dtype} maps={1 if lam is None else 2}")
        o, kept = ret.attention_fwd(q, k, v, lam, scale=USUAL, keep=True)
        gq, gk, gv, gl = ret.attention_bwd(q, k, v, o, do, kept, lam, scale=USUAL)
        qs, ks = q * a, k * b
        o2, kept2 = ret.attention_fwd(qs, ks, v, lam, scale=scale, keep=True)
        gq2, gk2, gv2, gl2 = ret.attention_bwd(qs, ks, v, o2, do, kept2, lam, scale=scale)
        assert torch.equal(o, o2) and torch.equal(kept[0], kept2[0]) and torch.equal(gv, gv2)
        assert lam is None or (torch.equal(kept[1], kept2[1]) and torch.equal(gl, gl2))
        assert torch.equal(gq, gq2 * a) and torch.equal(gk, gk2 * b)
        assert bool(gq.any()) and bool(gv.any())


@pytest.mark.parametrize("scale,a,b", ENDS)
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("most", [6, 400])
def test_decode_steps(most, dtype, scale, a, b):
    g = torch.Generator().manual_seed(most)
    B, H, Hk, dk, dv, page = 3, 4, 2, 64, 40, 16
    lens = torch.tensor([0, 37, 90], dtype=I32, device=DEV)
    table = torch.full((B, most), -1, dtype=I32)
    table[:, :6] = torch.randperm(B * 6, generator=g).view(B, 6).to(I32)
    q, k, kc = ints(g, B, H, dk, dtype=dtype), ints(g, B, Hk, dk, dtype=dtype), ints(g, B * 6, Hk, page, dk, dtype=dtype)
    v, vc = (torch.randn(s, generator=g).to(dtype).to(DEV) for s in ((B, Hk, dv), (B * 6, Hk, page, dv)))
    lam = torch.rand(H, generator=g).to(DEV)
    say(f"step at scale {scale:.3g}, {most} pages, {dtype}")
    want = ret.attention_step(q, k, v, kc.clone(), vc.clone(), table.to(DEV), lens, lam, scale=USUAL)
    got = ret.attention_step(q * a, k * b, v, kc * b, vc.clone(), table.to(DEV), lens, lam, scale=scale)
    assert torch.equal(want, got) and bool(got.any())


def test_small_scales_average_the_values():
    """Equal scores at the smallest scale: the mean of the values, with the keys split and not, and its gradient."""
    g = torch.Generator().manual_seed(1)
    for T, S in ((40, 40), (3, 1024)):
        q, k = torch.randn(1, 2, T, 32, generator=g).to(DEV), torch.randn(1, 2, S, 32, generator=g).to(DEV)
        v, do = torch.randn(1, 2, S, 16, generator=g).to(DEV), torch.randn(1, 2, T, 16, generator=g).to(DEV)
        o, kept = ret.attention_fwd(q, k, v, causal=False, scale=2.0 ** -100, keep=True)
        gv = ret.attention_bwd(q, k, v, o, do, kept, causal=False, scale=2.0 ** -100)[2]
        # S terms of 1 / S and T of do, in fp32
        assert (o.double() - v.double().mean(2, keepdim=True)).abs().max() <= (S + 8) * 2.0 ** -24 * float(v.abs().mean() * 2)
        assert (kept[0].double() - torch.tensor(float(S), dtype=torch.float64).log()).abs().max() <= 2.0 ** -20
        want = do.double().sum(2, keepdim=True) / S
        assert (gv.double() - want).abs().max() <= (T + 16) * 2.0 ** -22 * float(do.double().abs().sum(2).max()) / S
        with pytest.raises(ret.RetentionError, match="scale"):
            ret.attention_fwd(q, k, v, causal=False, scale=1e-38)

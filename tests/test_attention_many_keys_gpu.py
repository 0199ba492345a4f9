"""Sums over more keys of equal weight than fp32 counts one by one: 2^24 a lane, of four lanes a row."""
import math

import pytest
import torch

import retnet_retention_chunkwise_amd as ret
from helpers import say

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16, I32 = torch.bfloat16, torch.int32


def test_whole_sequences():
    """As many workgroups as fill the device, so that the keys are not split for its sake."""
    H, S = 256, (1 << 26) + (1 << 22)
    say(f"{S} keys, {H} heads")
    q = torch.zeros(1, H, 1, 1, dtype=BF16, device=DEV)
    k, v = torch.ones(1, 1, S, 1, dtype=BF16, device=DEV), torch.ones(1, 1, S, 1, dtype=BF16, device=DEV)
    o, (lse, _) = ret.attention_fwd(q, k, v, keep=True)
    torch.cuda.synchronize()
    assert (o == 1).all(), o.unique()
    # weights are 1 and every sum of them exact; a logarithm of 18 in fp32
    assert float((lse.double() - math.log(S)).abs().max()) <= 2.0 ** -19


def test_steps():
    """Full sequences that share one page; the new token is seen, not stored."""
    B, page, most = 512, 1 << 16, (1 << 12) + (1 << 8)
    say(f"{B} steps over {page * most} keys")
    q, k = torch.zeros(B, 1, 1, dtype=BF16, device=DEV), torch.ones(B, 1, 1, dtype=BF16, device=DEV)
    kc, vc = (torch.ones(1, 1, page, 1, dtype=BF16, device=DEV) for _ in range(2))
    table, lens = torch.zeros(B, most, dtype=I32, device=DEV), torch.full((B,), page * most, dtype=I32, device=DEV)
    o = ret.attention_step(q, k, torch.ones_like(k), kc, vc, table, lens)
    torch.cuda.synchronize()
    assert (o == 1).all(), o.unique()

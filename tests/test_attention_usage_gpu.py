"""Attention calls as programs make them: broadcast inputs, one workspace for all calls of a stream and of its graphs."""
import pytest
import torch

import retnet_retention_chunkwise_amd as ret
from helpers import say

pytestmark = pytest.mark.gpu

DEV = "cuda"
F32, BF16, I32 = torch.float32, torch.bfloat16, torch.int32


def rnd(g, *shape, dtype):
    return torch.randn(shape, generator=g).to(dtype).to(DEV)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_broadcast_inputs(dtype):
    """Keys and values of one prefix for all sequences, one gradient row for all tokens: the bits of copies."""
    B, H, Hk, T, S, d, dv = 3, 4, 2, 40, 90, 64, 48
    g = torch.Generator().manual_seed(1)
    say(f"broadcast {dtype}")
    q, lam = rnd(g, B, H, T, d, dtype=dtype), torch.rand(H, generator=g).to(DEV)
    k, v = rnd(g, 1, Hk, S, d, dtype=dtype).expand(B, -1, -1, -1), rnd(g, 1, Hk, S, dv, dtype=dtype).expand(B, -1, -1, -1)
    do = rnd(g, 1, 1, 1, dv, dtype=dtype).expand(B, H, T, dv)
    assert k.stride(0) == 0 and do.stride(2) == 0
    o, kept = ret.attention_fwd(q, k, v, lam, keep=True)
    got = (o, *kept, *ret.attention_bwd(q, k, v, o, do, kept, lam))
    kk, vv, dd = k.contiguous(), v.contiguous(), do.contiguous()
    o, kept = ret.attention_fwd(q, kk, vv, lam, keep=True)
    want = (o, *kept, *ret.attention_bwd(q, kk, vv, o, dd, kept, lam))
    assert all(a.shape == b.shape and torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_one_workspace_for_calls_and_graphs(dtype):
    """Calls of different sizes and two captured graphs that share a workspace, one after another on a stream."""
    g = torch.Generator().manual_seed(2)
    say(f"one workspace {dtype}")
    sets = []
    for T, S in ((300, 300), (8, 1500)):
        q, k, v, do = rnd(g, 1, 4, T, 64, dtype=dtype), rnd(g, 1, 2, S, 64, dtype=dtype), rnd(g, 1, 2, S, 64, dtype=dtype), rnd(
            g, 1, 4, T, 64, dtype=dtype)
        sets.append((q, k, v, torch.rand(4, generator=g).to(DEV), do))
    most = 80
    cache = [rnd(g, most, 2, 16, 64, dtype=dtype) for _ in range(2)]
    table, lens = torch.arange(most, dtype=I32, device=DEV)[None].contiguous(), torch.tensor([1200], dtype=I32, device=DEV)

    def all_of(i, ws):
        q, k, v, lam, do = sets[i]
        o, kept = ret.attention_fwd(q, k, v, lam, keep=True, workspace=ws)
        grads = ret.attention_bwd(q, k, v, o, do, kept, lam, workspace=ws)
        step = ret.attention_step(q[:, :, 0], k[:, :, 0], v[:, :, 0], *cache, table, lens, lam, workspace=ws)
        return (o, *kept, *grads, step)

    want = [all_of(i, None) for i in range(2)]
    ws = torch.full((1 << 25,), 255, dtype=torch.uint8, device=DEV)  # NaN in both types
    for i in (0, 1, 0):
        assert all(torch.equal(a, b) for a, b in zip(all_of(i, ws), want[i]))
    torch.cuda.synchronize()
    graphs = []
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            graphs.append((graph, all_of(i, ws)))
    for _ in range(3):
        for _, out in graphs:
            for t in out:
                t.fill_(float("nan"))
        for i in (1, 0):
            graphs[i][0].replay()
        all_of(0, ws)
        torch.cuda.synchronize()
        for (_, out), w in zip(graphs, want):
            assert all(torch.equal(a, b) for a, b in zip(out, w))
    small = torch.empty(1024, dtype=torch.uint8, device=DEV)
    q, k, v, lam, _ = sets[1]
    with pytest.raises((ValueError, ret.RetentionError), match="workspace"):
        ret.attention_fwd(q, k, v, lam, workspace=small)

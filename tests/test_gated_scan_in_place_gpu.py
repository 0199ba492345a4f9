"""The gated scan with its state in place (state_out is state_in, grad_state_in is grad_state_out) where a
channel run's tiles are worked on by several workgroups: the workgroup that writes the final state runs beside
others of the same run, and only the first tile may still be reading the incoming one.  In place and out of
place have to give the same bits, call after call, eagerly and in a captured graph."""
import pytest
import torch

import retnet_retention_chunkwise_amd as ret
from helpers import say

pytestmark = pytest.mark.gpu

DEV = "cuda"
# tiles of 64 channels by 128 tokens (16 channels by 512): 8 steps are the fewest that are chained
SIZES = [(1, 2, 1024, 64), (1, 1, 1025, 40), (2, 3, 3000, 64), (1, 2, 4096, 16), (3, 5, 1337, 201), (1, 8, 8250, 512)]


def inputs(B, H, T, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    t = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, dy, f = t(B, H, T, d), t(B, H, T, d), t(B, H, T, d) * 0.5 + 9  # long memories: the state reaches the end
    return [v.to(dtype).to(DEV) for v in (x, f, dy)] + [(10 * t(B, H, d)).to(DEV) for _ in range(2)]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,H,T,d", SIZES)
def test_state_in_place(B, H, T, d, dtype):
    say(f"scan in place B{B} H{H} T{T} d{d} {dtype}")
    x, f, dy, s, ds = inputs(B, H, T, d, dtype, B + T + d)
    rate = [2.0 ** -h for h in range(H)]
    assert ret.load().retention_gated_scan_workspace_bytes(B, H, T, d, int(dtype == torch.bfloat16)) > 0  # chained
    y, last, kept = ret.gated_scan_fwd(x, f, rate, s, normalize=True, checkpoints=True)
    gx, gf, gs = ret.gated_scan_bwd(x, f, rate, dy, s, ds, kept, True)
    # a call without a state is another: what enters has to count
    assert not torch.equal(last, ret.gated_scan_fwd(x, f, rate, normalize=True)[1])
    assert not torch.equal(gs, ret.gated_scan_bwd(x, f, rate, dy, s, None, kept, True)[2])
    state, grad = torch.empty_like(s), torch.empty_like(ds)

    def both():
        state.copy_(s)
        grad.copy_(ds)
        a = ret.gated_scan_fwd(x, f, rate, state, state_out=state, normalize=True, checkpoints=True)
        b = ret.gated_scan_bwd(x, f, rate, dy, None, grad, kept, True, grad_state_in=grad)
        assert a[1] is state and b[2] is grad
        return a[0], a[2], b[0], b[1]

    def check(got):
        for g, w in zip((*got, state, grad), (y, kept, gx, gf, last, gs)):
            assert torch.equal(g, w)

    for _ in range(5):
        check(both())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = both()
    for _ in range(5):
        for t in (*held, state, grad):
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        check(held)
        both()
        torch.cuda.synchronize()

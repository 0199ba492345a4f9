"""The gated scan over as many channel runs as a call may have, forward and backward, against the fp64 oracle at
sampled batch elements (bounds as derived in test_gated_scan_gpu)."""
import pytest
import torch

import retnet_retention_chunkwise_amd as ret
from helpers import say
from test_gated_scan_gpu import DEV, check_backward, check_forward, rates

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,H,T,d,dtype", [(4096, 32, 2, 512, torch.bfloat16), (1 << 18, 8, 1, 33, torch.float32)])
def test_many_runs(B, H, T, d, dtype):
    say(f"many runs B{B} H{H} T{T} d{d} {dtype}")
    g = torch.Generator(device=DEV).manual_seed(B + d)
    t = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    x, dy = t(B, H, T, d).to(dtype), t(B, H, T, d).to(dtype)
    f = (t(B, H, T, d) * 1.5 + 2).to(dtype)
    s, ds, rate = t(B, H, d), t(B, H, d), rates(H)
    y, last, kept = ret.gated_scan_fwd(x, f, rate, s, normalize=True, checkpoints=True)
    got = ret.gated_scan_bwd(x, f, rate, dy, s, ds, kept, True)
    pick = torch.tensor([0, 1, B // 3, B // 2 + 1, B - 2, B - 1], device=DEV)
    x, f, dy, s, ds = (v[pick].cpu() for v in (x, f, dy, s, ds))
    check_forward(f"many runs {B}", x, f, rate, s, True, y[pick], last[pick])
    check_backward(f"many runs {B}", x, f, rate, dy, s, ds, True, [v[pick] for v in got])

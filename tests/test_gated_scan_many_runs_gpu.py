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


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_one_token_has_no_stride_to_follow(dtype):
    """A dimension of one may have any stride; the backward of one token multiplies none of them."""
    B, H, d = 3, 2, 36
    g = torch.Generator().manual_seed(77)
    x, f, dy = (torch.randn(B, H, 1, d, generator=g).to(dtype) for _ in range(3))
    s, ds = torch.randn(B, H, d, generator=g), torch.randn(B, H, d, generator=g)

    def far(t):
        wide = torch.nn.functional.pad(t, (0, 4)).to(DEV)
        return wide.as_strided((B, H, 1, d), (H * (d + 4), d + 4, 2 ** 61, 1))

    out = lambda: far(torch.full((B, H, 1, d), float("nan"), dtype=dtype))  # noqa: E731
    got = ret.gated_scan_bwd(far(x), far(f), rates(H), far(dy), s.to(DEV), ds.to(DEV), None, True, grad_x=out(), grad_f=out())
    want = ret.gated_scan_bwd(*(t.to(DEV) for t in (x, f)), rates(H), dy.to(DEV), s.to(DEV), ds.to(DEV), None, True)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    check_backward("one token", x, f, rates(H), dy, s, ds, True, got)

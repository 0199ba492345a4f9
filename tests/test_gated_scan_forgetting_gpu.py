"""The gated scan where its gates forget: decays a far below 1, down to 0.

What the decay carries over is small there, and so is the gradient of its gate, but both have digits of their own:
they are held to bounds relative to a.  With u = 2^-24 and a = 2^(z2), z2 = -rate log2(1 + e^-f) in 32 bits:
z2 sums max(-f, 0) log2 e and log2(1 + t), t = e^-|f|; its constants, products and sum carry at most 16 u of z2, and
t, which is all of z2 where f > 0, 2 |f| u of itself.  So a carries at most
    ka u a,  ka = |z| (16 + 2 max(f, 0)) + 4,   z = ln a
(the exponential itself 4 u), and k = rate a sigmoid(-f) at most (ka + 2 max(f, 0) + 14) u more for t, the sum, the
reciprocal and the products.  An exponential below 2^-126 is 0: k may be off by (1 + rate) 2^-126.
"""
import pytest
import torch

import oracle
import retnet_retention_chunkwise_amd as ret
from helpers import rel_l2, say, tol
from test_gated_scan_gpu import DEV, F64, HALF, TINY, U, close, decays, h_bounds

pytestmark = pytest.mark.gpu

RATES = [1.0, 8.0, 0.25]
# walked, walked with a gate table (bf16), chained, chained and narrow
SIZES = [(2, 250, 40), (1, 700, 66), (1, 1500, 64), (1, 4500, 12)]


def forgetting(B, T, d, dtype, m, seed):
    """x, f, s, dy, ds with decays around e^-m (e^(-m/4) in the last head)."""
    g = torch.Generator().manual_seed(seed)
    t = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    H = len(RATES)
    f = 0.5 * t(B, H, T, d) - m / torch.tensor([max(r, 1.0) for r in RATES]).view(1, H, 1, 1)
    return t(B, H, T, d).to(dtype), f.to(dtype), t(B, H, d), t(B, H, T, d).to(dtype), t(B, H, d)


def ka_of(f, r):
    z = r * torch.logaddexp(torch.zeros_like(f), -f)
    return z * (16 + 2 * f.clamp(min=0)) + 4


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("m", [2, 6, 10, 14, 17, 24, 40])
def test_gradient_of_the_gate(m, normalize, dtype):
    """grad_f = g h' k with k = rate a sigmoid(-f): g and h' to the bounds of the recurrence, k relative to itself."""
    for B, T, d in SIZES:
        name = f"forgetting m={m} {dtype} normalize={normalize} T={T} d={d}"
        x, f, s, dy, ds = forgetting(B, T, d, dtype, m, T + m)
        X, F, S, DY, DS = (v.to(DEV) for v in (x, f, s, dy, ds))
        _, _, kept = ret.gated_scan_fwd(X, F, RATES, S, normalize=normalize, checkpoints=True)
        got = ret.gated_scan_bwd(X, F, RATES, DY, S, DS, kept, normalize)[1]
        want = oracle.gated_scan_backward(x, f, RATES, dy, s, ds, normalize)[1]
        before, eb, _ = h_bounds(x, f, RATES, s, normalize)
        x, f, dy = x.to(F64), f.to(F64), dy.to(F64)
        a, c, r = decays(f, RATES)
        k = a * r * torch.sigmoid(-f)
        kk = ka_of(f, r) + 2 * f.clamp(min=0) + 14
        ga, e = ds.to(F64).abs(), torch.zeros(B, len(RATES), d, dtype=F64)
        bound = torch.empty_like(x)
        for t in range(T - 1, -1, -1):
            at, ct, ft = a[:, :, t], c[:, :, t], f[:, :, t]
            g = dy[:, :, t].abs() + ga
            eg = e + 2 * U * g
            h = before[:, :, t] + (x[:, :, t].abs() if normalize else 0)
            tiny = (1 + r[:, :, 0]) * TINY
            bound[:, :, t] = k[:, :, t] * (eg * h + g * eb[:, :, t] + (kk[:, :, t] + 8) * U * g * h) + tiny * g * h
            e = at * eg + U * ((32 + 2 * ft.abs()) * ct * g + 6 * g) + tiny * g
            ga = at * g
        close(name + " grad_f", got, want, bound, HALF[dtype])
        err = rel_l2(got, want)
        say(f"{name}: rel-L2 {err:.2e}")
        assert err <= tol(dtype)

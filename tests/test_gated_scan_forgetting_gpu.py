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
    f = f.clamp(-1e4, 1e4)  # at f = -inf ka is infinite and a is 0, exactly: ka a counts as 0
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


# ---- the whole recurrence ----
#
# Bounds relative to what a leaves.  da: the error of a, ka u a below 1/2 (held as a) and (32 + 2 |f|) u c above
# (held as c = 1 - a; where a is next to 1/2 the larger one), and (1 + rate) 2^-126.  A step h' = a h + u rounds three
# times at most, at no more than the sum of magnitudes it forms, |h'| = a |h| + |u| (normalised and a < 1/2:
# x + a (h - x), where a |x| <= c |x|; else h + c (x - h), where c |h| <= a |h|).  A value that enters a thread's
# tokens has passed the maps of its segment, wave, tile and group: two roundings each, so 12 u of |h'| in all:
#     e' = a e + da (|h| + |x|) + 12 u |h'|.
# The same backwards: e(G) = a e(g) + da |g| + 12 u a |g| for G = a g, e(g) = e(G later) + 2 u |g|.
def h_tight(x, f, rate, s, normalize):
    """(|h| before every token, error bound there, error bound of every h) and the last."""
    x, f = x.to(F64), f.to(F64)
    a, c, r = decays(f, rate)
    da = U * torch.where(a < 0.45, ka_of(f, r) * a, (32 + 2 * f.abs().clamp(max=1e4)) * c) + (1 + r) * TINY
    ha = torch.zeros_like(x[:, :, 0]) if s is None else s.to(F64).abs()
    e = torch.zeros_like(ha)
    before, eb, err = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    for t in range(x.shape[2]):
        ax = x[:, :, t].abs()
        before[:, :, t], eb[:, :, t] = ha, e
        hn = a[:, :, t] * ha + (c[:, :, t] * ax if normalize else ax)
        e = a[:, :, t] * e + da[:, :, t] * (ha + ax) + 12 * U * hn
        ha = hn
        err[:, :, t] = e
    return before, eb, err, da


def check_tight(name, x, f, rate, s, dy, ds, normalize, y, last, got):
    h, hl = oracle.gated_scan(x, f, rate, s, normalize)
    want = oracle.gated_scan_backward(x, f, rate, dy, s, ds, normalize)
    before, eb, err, da = h_tight(x, f, rate, s, normalize)
    half = HALF[x.dtype]
    close(name + " y", y, h, err, half)
    close(name + " state", last, hl, err[:, :, -1], U)
    x, f, dy = x.to(F64), f.to(F64), dy.to(F64)
    a, c, r = decays(f, rate)
    k = a * r * torch.sigmoid(-f)
    kk = ka_of(f, r) + 2 * f.clamp(min=0) + 14
    ga = torch.zeros_like(x[:, :, 0]) if ds is None else ds.to(F64).abs()
    e = torch.zeros_like(ga)
    bx, bf = torch.empty_like(x), torch.empty_like(x)
    for t in range(x.shape[2] - 1, -1, -1):
        g = dy[:, :, t].abs() + ga
        eg = e + 2 * U * g
        m = before[:, :, t] + (x[:, :, t].abs() if normalize else 0)
        bx[:, :, t] = c[:, :, t] * eg + (da[:, :, t] + 2 * U * c[:, :, t]) * g if normalize else eg
        # the replayed h before a token has passed the maps too
        bf[:, :, t] = (k[:, :, t] * (eg * m + g * (eb[:, :, t] + 12 * U * m) + (kk[:, :, t] + 4) * U * g * m)
                       + (1 + r[:, :, 0]) * TINY * g * m)
        e = a[:, :, t] * eg + da[:, :, t] * g + 12 * U * a[:, :, t] * g
        ga = a[:, :, t] * g
    close(name + " grad_x", got[0], want[0], bx, half)
    close(name + " grad_f", got[1], want[1], bf, half)
    close(name + " grad_state", got[2], want[2], e, U)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("m", [1, 2, 6, 10, 17, 40])
def test_a_large_past_is_forgotten(m, normalize, dtype):
    """A carried state and a gradient behind of 1e6: what the gates leave of them counts, not their rounding."""
    for B, T, d in SIZES:
        name = f"large past m={m} {dtype} normalize={normalize} T={T} d={d}"
        x, f, s, dy, ds = forgetting(B, T, d, dtype, m, T + m)
        s, ds = 1e6 * s, 1e6 * ds
        x[:, :, T // 2] *= 1e4  # and a token of large values amid the others
        X, F, S, DY, DS = (v.to(DEV) for v in (x, f, s, dy, ds))
        y, last, kept = ret.gated_scan_fwd(X, F, RATES, S, normalize=normalize, checkpoints=True)
        got = ret.gated_scan_bwd(X, F, RATES, DY, S, DS, kept, normalize)
        check_tight(name, x, f, RATES, s, dy, ds, normalize, y, last, got)
        state = S.clone()
        n = min(T, 6)
        ys = [ret.gated_scan_step(X[:, :, t], F[:, :, t], RATES, state, normalize) for t in range(n)]
        h, hl = oracle.gated_scan(x[:, :, :n], f[:, :, :n], RATES, s, normalize)
        err = h_tight(x[:, :, :n], f[:, :, :n], RATES, s, normalize)[2]
        close(name + " steps", torch.stack(ys, 2), h, err, HALF[dtype])
        close(name + " stepped state", state, hl, err[:, :, -1], U)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("size", [1e4, 1e8])
def test_a_reset_starts_anew(size, normalize, dtype):
    """After f = -inf nothing is left of a state of 1e4 or 1e8, not even its rounding: the token is x exactly, and
    what follows is held to the bounds of a sequence that starts there; the step likewise."""
    for B, T, d in SIZES:
        name = f"reset {size:g} {dtype} normalize={normalize} T={T} d={d}"
        say(name)
        x, f, s, dy, ds = forgetting(B, T, d, dtype, 0, T)
        at = torch.full((T,), False)
        at[[0, 1, 37, 120, T // 2, T - 2]] = True
        f[:, :, at] = -torch.inf
        before = (at.nonzero().flatten() - 1).clamp(min=0)
        x[:, :, before[~at[before]]] *= size  # so that every reset but the second has a large value before it
        s = s * size
        X, F, S = (v.to(DEV) for v in (x, f, s))
        y, last = ret.gated_scan_fwd(X, F, RATES, S, normalize=normalize)
        assert torch.equal(y[:, :, at.to(DEV)], X[:, :, at.to(DEV)])
        ends = at.nonzero().flatten().tolist() + [T]
        for t0, t1 in zip(ends, ends[1:]):
            part = x[:, :, t0:t1], f[:, :, t0:t1]
            close(f"{name} from {t0}", y[:, :, t0:t1], oracle.gated_scan(*part, RATES, None, normalize)[0],
                  h_tight(*part, RATES, None, normalize)[2], HALF[dtype])
        state = S.clone()
        y1 = ret.gated_scan_step(X[:, :, 0], F[:, :, 0], RATES, state, normalize)
        assert torch.equal(y1, X[:, :, 0]) and torch.equal(state, X[:, :, 0].float())


def every_gate(dtype):
    """All finite bf16 values; in fp32 as many spread over -100..100, and around where 1 + e^-f rounds to 1."""
    if dtype == torch.bfloat16:
        v = torch.arange(-2 ** 15, 2 ** 15, dtype=torch.int32).to(torch.int16).view(torch.bfloat16)
        v = v[torch.isfinite(v)]
        return torch.cat([v, v.new_zeros(2 ** 16 - len(v))])
    n = 2 ** 15
    return torch.cat([torch.linspace(-100, 100, n), torch.linspace(13, 20, n)])


@pytest.mark.parametrize("rate", [1.0, 1 / 16, 3.0, 40.0])
@pytest.mark.parametrize("T", [1, 40, 300])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_every_gate(dtype, T, rate):
    """One token with each gate among tokens that keep the state (f = inf, x = 0): from a state of 1 and x = 0 the
    output is a, from no state and x = 1 it is 1 - a (normalised); directly and by table."""
    f1 = every_gate(dtype).view(128, 1, 512)
    t0 = T // 3
    f = torch.full((128, 1, T, 512), torch.inf, dtype=dtype)
    f[:, :, t0] = f1
    F = f.to(DEV)
    x = torch.zeros_like(F)
    one = torch.ones(128, 1, 512, device=DEV)
    _, a = ret.gated_scan_fwd(x, F, [rate], one)
    _, an = ret.gated_scan_fwd(x, F, [rate], one, normalize=True)
    x[:, :, t0] = 1.0
    _, c = ret.gated_scan_fwd(x, F, [rate], normalize=True)
    va, vc, r = decays(f1.unsqueeze(2).to(F64), [rate])
    va, vc, vf = va.squeeze(2), vc.squeeze(2), f1.to(F64)
    da = U * torch.where(va < 0.45, ka_of(vf, rate) * va, (32 + 2 * vf.abs().clamp(max=1e4)) * vc) + (1 + rate) * TINY
    name = f"every gate {dtype} T={T} rate={rate}"
    close(name + " a", a, va, da, 2 * U)
    close(name + " a, normalised", an, va, da, 2 * U)
    close(name + " 1 - a", c, vc, torch.where(va < 0.45, da, U * (32 + 2 * vf.abs().clamp(max=1e4)) * vc + (1 + rate) * TINY),
          2 * U)

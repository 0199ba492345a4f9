"""GPU parity of the gated GroupNorm and the residual norm (forward and
backward) against the fp64 CPU oracle, element by element, and of a block that
runs the gated scan, both norms and the retention operators together.

Bounds, u = 2^-24.  A row sum adds at most 16 values in a thread, 6 wave steps
and 16 wave sums: its error is within 36 u of the sum of magnitudes.  So the
mean is off by 36 u mean|y| and xh = (y - mu) rstd by
    E = 36 u rstd (mean|y| + |y|) + 40 u |xh|
(the variance is a sum about the mean: 36 u + 2 u of it, half of that for rstd,
and its square root, reciprocal and products at most 20 u more).
sigmoid(z) carries (|z| + 6) u (the product z log2 e, the exponential, the sum,
the reciprocal), and nothing below 2^-126.  A sum over N rows of one parameter
adds N u of its magnitudes.  Rounding to bf16 adds 2^-8 of the value.
"""
import math

import pytest
import torch

import oracle
import retnet_retention_chunkwise_amd as ret
from helpers import F32_TOL, rel_l2, say

pytestmark = pytest.mark.gpu

DEV, F64, U, TINY = "cuda", torch.float64, 2.0 ** -24, 2.0 ** -126
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
EPS = 1e-5


def rnd(g, *shape, dtype=torch.float32, scale=1.0, shift=0.0):
    return (torch.randn(shape, generator=g) * scale + shift).to(dtype)


def close(name, got, want, bound, half):
    got, want = got.detach().cpu().to(F64), want.to(F64)
    lim = bound + half * want.abs() + 1e-37
    worst = float(((got - want).abs() / lim).max()) if got.numel() else 0.0
    say(f"{name}: worst error {worst:.3f} of its bound")
    assert got.shape == want.shape and torch.isfinite(got).all() and worst <= 1.0, (name, worst)


def up(t):
    return None if t is None else t.detach().cpu().to(F64)


def hat(y, eps, center=True):
    """(xh, rstd, error bound of xh) of rows in fp64."""
    mu = y.mean(-1, keepdim=True) if center else torch.zeros_like(y[..., :1])
    rstd = 1 / torch.sqrt(((y - mu) ** 2).mean(-1, keepdim=True) + eps)
    xh = (y - mu) * rstd
    return xh, rstd, 36 * U * rstd * (y.abs().mean(-1, keepdim=True) + y.abs()) + 40 * U * xh.abs()


def norm_bwd_bound(xh, rstd, e, p, ep, center):
    """Error bound of rstd (p - mean p - xh mean(p xh)) for errors e of xh and ep of p."""
    ap, ax = p.abs(), xh.abs()
    mpx = (p * xh).mean(-1, keepdim=True).abs()
    empx = (ep * ax + ap * e + 40 * U * ap * ax).mean(-1, keepdim=True)
    emp = (ep + 40 * U * ap).mean(-1, keepdim=True) if center else 0.0
    size = ap + (ap.mean(-1, keepdim=True) if center else 0.0) + ax * (ap * ax).mean(-1, keepdim=True)
    return rstd * (ep + emp + ax * empx + e * mpx + 30 * U * size)


# ----------------------------------------------------------- gated GroupNorm
def gate_parts(z):
    s = torch.sigmoid(z)
    ks = (z.abs() + 10) * U
    return z * s, (z.abs() * s) * ks + z.abs() * TINY, s + z * s * (1 - s), (1 + z.abs()) * (s * ks + 2 * U * s + TINY)


def check_gate_fwd(name, y, z, w, b, got, eps=EPS):
    xh, rstd, e = hat(up(y), eps)
    want = oracle.group_norm_gated(y, z, w, b, eps)
    ww = torch.ones_like(xh) if w is None else up(w)[:, None]
    bb = torch.zeros_like(xh) if b is None else up(b)[:, None]
    n = xh * ww + bb
    en = (e * ww.abs() + 3 * U * ((xh * ww).abs() + bb.abs())).transpose(1, 2)
    if z is not None:
        sg, esg, _, _ = gate_parts(up(z))
        en = en * sg.abs() + n.transpose(1, 2).abs() * (esg + 2 * U * sg.abs())
    close(name, got, want, en, HALF[y.dtype])


def check_gate_bwd(name, y, z, do, w, b, got, eps=EPS):
    B, H, T, dv = y.shape
    xh, rstd, e = hat(up(y), eps)
    want = oracle.group_norm_gated_backward(y, z, do, w, b, eps)
    ww = torch.ones_like(xh) if w is None else up(w)[:, None]
    bb = torch.zeros_like(xh) if b is None else up(b)[:, None]
    d = up(do).transpose(1, 2)
    dn, edn = d, torch.zeros_like(d)
    if z is not None:
        sg, esg, ds, eds = gate_parts(up(z).transpose(1, 2))
        dn, edn = d * sg, d.abs() * (esg + 2 * U * sg.abs())
        n = xh * ww + bb
        en = e * ww.abs() + 3 * U * ((xh * ww).abs() + bb.abs())
        ez = d.abs() * (n.abs() * eds + ds.abs() * en + 3 * U * (n * ds).abs())
        close(name + " grad_gate", got[1], want[1], ez.transpose(1, 2), HALF[y.dtype])
    else:
        assert got[1] is None
    p, ep = dn * ww, edn * ww.abs() + 2 * U * (dn * ww).abs()
    close(name + " grad_y", got[0], want[0], norm_bwd_bound(xh, rstd, e, p, ep, True), HALF[y.dtype])
    N = B * T
    for k, (g, ref, err, size) in enumerate(((got[2], want[2], dn.abs() * e + edn * xh.abs(), (dn * xh).abs()),
                                             (got[3], want[3], edn, dn.abs()))):
        if (w, b)[k] is None:
            assert g is None
        else:
            close(name + (" grad_weight", " grad_bias")[k], g, ref, (err + (N + 4) * U * size).sum((0, 2)), U)


GATE_CASES = [
    # B, H, T, dv, dtype, gate, weight, bias
    (1, 1, 1, 1, torch.float32, True, True, True),
    (2, 3, 5, 7, torch.bfloat16, True, True, True),
    (1, 2, 33, 8, torch.bfloat16, True, False, False),
    (3, 2, 17, 64, torch.float32, True, True, False),
    (2, 5, 40, 72, torch.bfloat16, False, True, True),
    (1, 3, 130, 128, torch.bfloat16, True, True, True),
    (2, 2, 31, 201, torch.float32, True, True, True),
    (1, 4, 300, 256, torch.bfloat16, True, False, True),
    (2, 2, 65, 260, torch.float32, False, False, False),
    (128, 16, 1, 512, torch.bfloat16, True, True, True),
    (1, 2, 700, 511, torch.float32, True, True, True),
    (2, 1300, 2, 16, torch.float32, True, True, True),
]


@pytest.mark.parametrize("B,H,T,dv,dtype,gate,weight,bias", GATE_CASES)
def test_gate_norm_matches_oracle(B, H, T, dv, dtype, gate, weight, bias):
    name = f"gate norm B{B} H{H} T{T} dv{dv} {dtype} gate={gate} weight={weight} bias={bias}"
    say(name)
    g = torch.Generator().manual_seed(B + H + T + dv)
    y = rnd(g, B, H, T, dv, dtype=dtype, scale=0.5, shift=0.7)
    z = rnd(g, B, T, H, dv, dtype=dtype, scale=2) if gate else None
    w, b = rnd(g, H, dv, shift=1) if weight else None, rnd(g, H, dv) if bias else None
    do = rnd(g, B, T, H, dv, dtype=dtype)
    dev = [None if t is None else t.to(DEV) for t in (y, z, w, b, do)]
    out = ret.group_norm_gated(dev[0], dev[1], dev[2], dev[3], EPS)
    check_gate_fwd(name, y, z, w, b, out)
    got = ret.group_norm_gated_bwd(dev[0], dev[1], dev[4], dev[2], dev[3], EPS)
    check_gate_bwd(name, y, z, do, w, b, got)
    again = ret.group_norm_gated_bwd(dev[0], dev[1], dev[4], dev[2], dev[3], EPS)
    assert all(p is q or torch.equal(p, q) for p, q in zip(got, again))
    bare = ret.group_norm_gated_bwd(dev[0], dev[1], dev[4], dev[2], dev[3], EPS, param_grads=False)
    assert bare[2] is None and bare[3] is None and torch.equal(bare[0], got[0])


def test_gate_norm_without_gate_is_group_norm():
    g = torch.Generator().manual_seed(5)
    y, w, b = rnd(g, 2, 4, 50, 256, dtype=torch.bfloat16).to(DEV), rnd(g, 4, 256).to(DEV), rnd(g, 4, 256).to(DEV)
    out = ret.group_norm_gated(y, None, w, b)
    assert rel_l2(out.transpose(1, 2), ret.group_norm(y, w, b)) <= 2.0 ** -8  # each rounds once


NARROW = [(B, H, T, dv, dt) for B, H, T in ((1, 1, 1), (2, 3, 67), (3, 2, 700))
          for dv in (1, 3, 4, 7, 8, 9, 15, 16, 25, 31, 32, 33) for dt in (torch.float32, torch.bfloat16)]


@pytest.mark.parametrize("B,H,T,dv,dtype", NARROW)
def test_gate_norm_of_narrow_heads(B, H, T, dv, dtype):
    test_gate_norm_matches_oracle(B, H, T, dv, dtype, True, True, True)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dv", [64, 40, 33])
def test_gate_norm_layouts_and_untouched_surroundings(dtype, dv):
    """A gate that is a slice of a fused projection, outputs into wider buffers, y in either order."""
    B, H, T = 2, 3, 21
    g = torch.Generator().manual_seed(6)
    y, z = rnd(g, B, H, T, dv, dtype=dtype), rnd(g, B, T, H, dv, dtype=dtype)
    w, b, do = rnd(g, H, dv, shift=1), rnd(g, H, dv), rnd(g, B, T, H, dv, dtype=dtype)
    W = H * dv
    fused = torch.full((B, T + 2, 3 * W + 5), 7.0, dtype=dtype, device=DEV)
    zs = fused[:, :T, W:2 * W].unflatten(-1, (H, dv))
    zs.copy_(z)
    ys = torch.empty(B, T, H, dv, dtype=dtype, device=DEV).transpose(1, 2)
    ys.copy_(y)
    buf = torch.full((B, T + 2, 3 * W + 5), 7.0, dtype=dtype, device=DEV)
    out = buf[:, :T, 1:W + 1].unflatten(-1, (H, dv))
    got = ret.group_norm_gated(ys, zs, w.to(DEV), b.to(DEV), EPS, out=out)
    assert got is out
    check_gate_fwd(f"strided gate norm dv{dv} {dtype}", y, z, w, b, out)
    out.fill_(7.0)
    assert torch.equal(buf, torch.full_like(buf, 7.0))
    gz = buf[:, :T, W:2 * W].unflatten(-1, (H, dv))
    gy = buf[:, :T, 2 * W + 3:3 * W + 3].unflatten(-1, (H, dv)).transpose(1, 2)
    grads = ret.group_norm_gated_bwd(ys, zs, do.to(DEV), w.to(DEV), b.to(DEV), EPS, grad_y=gy, grad_gate=gz)
    check_gate_bwd(f"strided gate norm dv{dv} {dtype}", y, z, do, w, b, grads)
    gz.fill_(7.0)
    gy.fill_(7.0)
    assert torch.equal(buf, torch.full_like(buf, 7.0))


def test_gate_norm_hard_rows():
    """Constant rows, a mean far from zero, tiny and large rows, gates up to the type's limits."""
    dv = 128
    g = torch.Generator().manual_seed(7)
    y = rnd(g, 1, 1, 8, dv)
    y[0, 0, 0] = 3.0
    y[0, 0, 1] = 0.0
    y[0, 0, 2] += 1000.0
    y[0, 0, 3] *= 1e-12
    y[0, 0, 4] *= 1e12
    y[0, 0, 5, 7] = 1e4
    z = rnd(g, 1, 8, 1, dv, scale=3)
    z[0, 6, 0, :8] = torch.tensor([200.0, -200.0, 88.0, -88.0, 3e38, -3e38, 0.0, -0.0])
    z[0, 7] = -torch.finfo(torch.float32).max
    w, b, do = rnd(g, 1, dv, shift=1), rnd(g, 1, dv), rnd(g, 1, 8, 1, dv)
    out = ret.group_norm_gated(y.to(DEV), z.to(DEV), w.to(DEV), b.to(DEV), EPS)
    check_gate_fwd("hard rows", y, z, w, b, out)
    z[0, 6, 0, 4] = 300.0  # the gradient of a product with 3e38 leaves the type's range
    got = ret.group_norm_gated_bwd(y.to(DEV), z.to(DEV), do.to(DEV), w.to(DEV), b.to(DEV), EPS)
    check_gate_bwd("hard rows", y, z, do, w, b, got)


def test_gate_norm_bad_row_stays_alone():
    g = torch.Generator().manual_seed(8)
    y, z = rnd(g, 2, 3, 9, 40).to(DEV), rnd(g, 2, 9, 3, 40).to(DEV)
    clean = ret.group_norm_gated(y, z)
    cg = ret.group_norm_gated_bwd(y, z, z)
    for bad in (math.nan, math.inf):
        yy = y.clone()
        yy[1, 2, 4, 5] = bad
        out = ret.group_norm_gated(yy, z)
        gy, gz, _, _ = ret.group_norm_gated_bwd(yy, z, z)
        keep = torch.ones(2, 9, 3, dtype=torch.bool, device=DEV)
        keep[1, 4, 2] = False
        assert torch.equal(out[keep], clean[keep]) and torch.isnan(out[~keep]).all()
        assert torch.equal(gz[keep], cg[1][keep]) and torch.equal(gy.transpose(1, 2)[keep], cg[0].transpose(1, 2)[keep])


def test_gate_norm_empty():
    y, w = torch.empty(2, 3, 0, 8, device=DEV), torch.ones(3, 8, device=DEV)
    z = torch.empty(2, 0, 3, 8, device=DEV)
    assert ret.group_norm_gated(y, z, w, w).shape == z.shape
    gy, gz, gw, gb = ret.group_norm_gated_bwd(y, z, z, w, w)
    assert gy.shape == y.shape and gz.shape == z.shape and not gw.any() and not gb.any()


# ------------------------------------------------------------- residual norm
def check_residual(name, x, f, w, b, s, alpha, rms, r, n):
    want = oracle.residual(x, f, s, alpha)
    size = (alpha * up(x)).abs() + (up(f) if s is None else up(s) * up(f)).abs()
    close(name + " r", r, want, 3 * U * size, HALF[x.dtype])
    held = up(r)  # the norm is of the stream as it is stored
    xh, rstd, e = hat(held, EPS, not rms)
    ww = torch.ones_like(xh) if w is None else up(w)
    bb = torch.zeros_like(xh) if b is None else up(b)
    close(name + " n", n, oracle.stream_norm(held, w, b, EPS, rms),
          e * ww.abs() + 3 * U * ((xh * ww).abs() + bb.abs()), HALF[x.dtype])


def check_residual_bwd(name, r, dn, dr, w, f, s, alpha, rms, got):
    want = oracle.residual_norm_backward(r, dn, dr, w, f, s, alpha, EPS, rms)
    xh, rstd, e = hat(up(r), EPS, not rms)
    p = up(dn) if w is None else up(dn) * up(w)
    g = want[0] / alpha
    eg = norm_bwd_bound(xh, rstd, e, p, 2 * U * p.abs(), not rms) + 3 * U * (g.abs() + (0 if dr is None else up(dr).abs()))
    sc = torch.ones_like(xh) if s is None else up(s).expand_as(xh)
    close(name + " grad_x", got[0], want[0], abs(alpha) * (eg + 2 * U * g.abs()), HALF[r.dtype])
    close(name + " grad_f", got[1], want[1], sc.abs() * (eg + 2 * U * g.abs()), HALF[r.dtype])
    N = r.numel() // r.shape[-1]
    rows = tuple(range(r.dim() - 1))
    if got[2] is not None:
        d = up(dn).abs()
        close(name + " grad_weight", got[2], want[2], (d * e + (N + 4) * U * (d * xh.abs())).sum(rows), U)
    if got[3] is not None:
        close(name + " grad_bias", got[3], want[3], ((N + 4) * U * up(dn).abs()).sum(rows), U)
    if got[4] is not None:
        af = up(f).abs()
        close(name + " grad_scale", got[4], want[4], (eg * af + (N + 4) * U * g.abs() * af).sum(rows), U)


RES_CASES = [
    # rows, D, dtype, rms, weight, bias, scale, alpha
    (1, 1, torch.float32, False, True, True, True, 1.0),
    (3, 5, torch.bfloat16, True, True, False, False, 1.0),
    (37, 64, torch.bfloat16, False, True, True, False, 1.0),
    (200, 72, torch.float32, True, False, False, True, 0.5),
    (9, 130, torch.bfloat16, False, True, True, True, 1.7),
    (300, 255, torch.float32, False, False, False, False, 2.0),
    (65, 512, torch.bfloat16, True, True, False, True, 1.0),
    (77, 1000, torch.bfloat16, False, True, True, True, 1.0),
    (130, 1111, torch.float32, True, True, False, True, 1.5),
    (128, 2048, torch.bfloat16, False, True, True, False, 1.0),
    (33, 4096, torch.float32, False, True, True, True, 1.0),
    (600, 4096, torch.bfloat16, True, True, False, True, 1.0),
    (17, 8192, torch.bfloat16, False, True, True, True, 1.0),
    (5, 8191, torch.bfloat16, True, True, False, False, 0.1),
    (9, 12288, torch.bfloat16, False, True, True, True, 1.0),
    (3, 16384, torch.float32, True, True, True, True, 1.0),
    (2, 16383, torch.float32, False, True, True, True, 1.0),
    (5000, 24, torch.float32, False, True, True, True, 1.0),
]


@pytest.mark.parametrize("rows,D,dtype,rms,weight,bias,scale,alpha", RES_CASES)
def test_residual_norm_matches_oracle(rows, D, dtype, rms, weight, bias, scale, alpha):
    name = f"residual norm rows{rows} D{D} {dtype} rms={rms} w={weight} b={bias} s={scale} alpha={alpha}"
    say(name)
    g = torch.Generator().manual_seed(rows + D)
    x, f = rnd(g, rows, D, dtype=dtype, scale=2, shift=0.5), rnd(g, rows, D, dtype=dtype)
    w, b = rnd(g, D, shift=1) if weight else None, rnd(g, D) if bias else None
    s = rnd(g, D) if scale else None
    dev = [None if t is None else t.to(DEV) for t in (x, f, w, b, s)]
    r, n = ret.residual_norm(dev[0], dev[1], dev[2], dev[3], dev[4], alpha, EPS, rms)
    check_residual(name, x, f, w, b, s, alpha, rms, r, n)
    dn, dr = rnd(g, rows, D, dtype=dtype), rnd(g, rows, D, dtype=dtype)
    for d in (dr, None):
        args = (r, dn.to(DEV), None if d is None else d.to(DEV), dev[2], dev[1], dev[4], alpha, EPS, rms, bias)
        got = ret.residual_norm_bwd(*args)
        check_residual_bwd(name, r, dn, d, w, f, s, alpha, rms, got)
        again = ret.residual_norm_bwd(*args)
        assert all(p is q or torch.equal(p, q) for p, q in zip(got, again))
    bare = ret.residual_norm_bwd(r, dn.to(DEV), None, dev[2], None, dev[4], alpha, EPS, rms, param_grads=False)
    assert bare[2] is None and bare[3] is None and bare[4] is None and torch.equal(bare[0], got[0])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D", [64, 33, 1000])
def test_residual_norm_layouts_and_untouched_surroundings(dtype, D):
    B, T = 3, 11
    g = torch.Generator().manual_seed(9)
    x, f = rnd(g, B, T, D, dtype=dtype), rnd(g, B, T, D, dtype=dtype)
    wide = torch.full((B, T, 2 * D + 3), 7.0, dtype=dtype, device=DEV)
    xs, fs = wide[..., :D], wide[..., D + 1:2 * D + 1]
    xs.copy_(x)
    fs.copy_(f)
    buf = torch.full((B, T, 2 * D + 3), 7.0, dtype=dtype, device=DEV)
    r, n = ret.residual_norm(xs, fs, r=buf[..., 1:D + 1], n=buf[..., D + 2:2 * D + 2])
    check_residual(f"strided residual norm D{D} {dtype}", x, f, None, None, None, 1.0, False, r, n)
    dn = wide[..., D + 1:2 * D + 1]
    got = ret.residual_norm_bwd(r, dn, xs)
    check_residual_bwd(f"strided residual norm D{D} {dtype}", r, f, x, None, None, None, 1.0, False, got)
    assert got[0] is got[1]
    r.fill_(7.0)
    n.fill_(7.0)
    assert torch.equal(buf, torch.full_like(buf, 7.0))
    with pytest.raises(ValueError, match="evenly"):
        ret.residual_norm(wide[:, :5, :D], wide[:, :5, :D])


def test_residual_norm_hard_rows():
    D = 320
    g = torch.Generator().manual_seed(10)
    x, f = rnd(g, 6, D), rnd(g, 6, D)
    x[0], f[0] = 5.0, -5.0
    x[1], f[1] = 2.0, 1.0
    x[2] += 1e5
    x[3, 3] = 1e6
    x[4] *= 1e-15
    f[4] *= 1e-15
    for rms in (False, True):
        r, n = ret.residual_norm(x.to(DEV), f.to(DEV), rms=rms)
        check_residual(f"hard rows rms={rms}", x, f, None, None, None, 1.0, rms, r, n)
        got = ret.residual_norm_bwd(r, f.to(DEV), x.to(DEV), rms=rms)
        check_residual_bwd(f"hard rows rms={rms}", r, f, x, None, None, None, 1.0, rms, got)


def test_residual_norm_empty():
    x, w = torch.empty(0, 8, device=DEV), torch.ones(8, device=DEV)
    r, n = ret.residual_norm(x, x, w, w)
    assert r.shape == x.shape and n.shape == x.shape
    gx, gf, gw, gb, gs = ret.residual_norm_bwd(x, x, x, w, x, w, bias_grad=True)
    assert not gw.any() and not gb.any() and not gs.any()


def test_norm_bindings_refuse():
    y, z = torch.randn(2, 3, 4, 8, device=DEV), torch.randn(2, 4, 3, 8, device=DEV)
    w = torch.ones(3, 8, device=DEV)
    x = torch.randn(6, 8, device=DEV)
    for bad in (lambda: ret.group_norm_gated(y, z.bfloat16()), lambda: ret.group_norm_gated(y, y),
                lambda: ret.group_norm_gated(y, z, w.bfloat16()), lambda: ret.group_norm_gated(y, z, w[:2]),
                lambda: ret.group_norm_gated(y, z, out=z), lambda: ret.group_norm_gated(y, z, eps=-1.0),
                lambda: ret.group_norm_gated(torch.randn(1, 1, 2, 513, device=DEV)),
                lambda: ret.group_norm_gated(y.cpu(), z.cpu()), lambda: ret.group_norm_gated_bwd(y, z, y),
                lambda: ret.group_norm_gated_bwd(y, z, z, grad_gate=z), lambda: ret.residual_norm(x, x[:3]),
                lambda: ret.residual_norm(x, x, torch.ones(7, device=DEV)), lambda: ret.residual_norm(x, x, r=x),
                lambda: ret.residual_norm(x, x, alpha=math.inf), lambda: ret.residual_norm(x.half(), x.half()),
                lambda: ret.residual_norm(torch.randn(1, 16385, device=DEV), torch.randn(1, 16385, device=DEV)),
                lambda: ret.residual_norm_bwd(x, x, x, scale=torch.ones(8, device=DEV))):
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            bad()


# --------------------------------------------------------------- a whole block
def _block(x, res, p, rate, C, f32_ref=False):
    """Retention and a gated scan side by side, gated norm of their sum's parts, and the residual: forward and
    the gradients of every input for given output gradients, through the library."""
    q, k, v, f, gate = x
    gamma, w, b, wn, scale, dr, dn = p
    y1, _ = ret.chunkwise_fwd(q, k, v, gamma, C)
    y2, _, kept = ret.gated_scan_fwd(v, f, rate, normalize=True, checkpoints=True)
    o1 = ret.group_norm_gated(y1, gate, w, b)
    o2 = ret.group_norm_gated(y2, gate, w, b)
    B, T, H, dv = o1.shape
    r1, _ = ret.residual_norm(res, o1.reshape(B, T, H * dv), wn, scale=scale, rms=True)
    r2, n = ret.residual_norm(r1, o2.reshape(B, T, H * dv), wn, scale=scale, rms=True)
    g2, go2, gw2, _, gs2 = ret.residual_norm_bwd(r2, dn, dr, wn, o2.reshape(B, T, H * dv), scale, rms=True)
    g1, go1, gs1 = g2, g2 * scale.to(g2.dtype), (g2 * o1.reshape(B, T, H * dv)).sum((0, 1))
    gy2, gg2, gwn2, gb2 = ret.group_norm_gated_bwd(y2, gate, go2.view(B, T, H, dv), w, b)
    gy1, gg1, gwn1, gb1 = ret.group_norm_gated_bwd(y1, gate, go1.view(B, T, H, dv), w, b)
    gv2, gf, _ = ret.gated_scan_bwd(v, f, rate, gy2, checkpoints=kept, normalize=True)
    gq, gk, gv1, _ = ret.chunkwise_bwd(q, k, v, gamma, C, gy1)
    return (r2, n), (gq, gk, gv1 + gv2, gf, gg1 + gg2, g1, gwn1 + gwn2, gb1 + gb2, gw2, gs1 + gs2)


def test_block_runs_together():
    """Retention and the gated scan, each through the gated norm, added to a stream: outputs and the gradient of
    every input and parameter against fp64 autograd of the written-out formulas (32-bit inputs)."""
    B, H, T, dk, dv, C = 2, 2, 150, 16, 24, 32
    g = torch.Generator().manual_seed(40)
    q, k = rnd(g, B, H, T, dk, scale=0.25), rnd(g, B, H, T, dk, scale=0.25)
    v, f = rnd(g, B, H, T, dv), rnd(g, B, H, T, dv, shift=1)
    gate, res = rnd(g, B, T, H, dv), rnd(g, B, T, H * dv)
    w, b, wn, scale = rnd(g, H, dv, shift=1), rnd(g, H, dv), rnd(g, H * dv, shift=1), rnd(g, H * dv)
    dr, dn = rnd(g, B, T, H * dv), rnd(g, B, T, H * dv)
    gamma, rate = [0.9, 0.97], [1.0, 0.25]
    d = lambda *ts: [t.to(DEV) for t in ts]  # noqa: E731
    outs, grads = _block(d(q, k, v, f, gate), res.to(DEV), [gamma, *d(w, b, wn, scale, dr, dn)], rate, C)

    leaves = [t.to(F64).requires_grad_() for t in (q, k, v, f, gate, res, w, b, wn, scale)]
    Q, K, V, F, Z, R, W, Bb, WN, S = leaves
    i = torch.arange(T)
    mask = torch.stack([torch.tril(torch.tensor(gm, dtype=torch.float32).to(F64) ** (i[:, None] - i[None]).clamp(min=0))
                        for gm in gamma])
    y1 = ((Q @ K.transpose(-1, -2)) * mask) @ V
    loga = torch.nn.functional.logsigmoid(F) * torch.tensor(rate, dtype=F64).view(1, -1, 1, 1)
    h, y2 = torch.zeros(B, H, dv, dtype=F64), []
    for t in range(T):
        h = torch.exp(loga[:, :, t]) * h + -torch.expm1(loga[:, :, t]) * V[:, :, t]
        y2.append(h)
    y2 = torch.stack(y2, 2)

    def gated(y):
        n = torch.nn.functional.layer_norm(y, (dv,), eps=1e-5) * W[:, None] + Bb[:, None]
        return (n.transpose(1, 2) * torch.nn.functional.silu(Z)).reshape(B, T, H * dv)

    r2 = R + S * gated(y1) + S * gated(y2)
    n = r2 * torch.rsqrt((r2 ** 2).mean(-1, keepdim=True) + 1e-5) * WN
    want = torch.autograd.grad((r2 * dr.to(F64)).sum() + (n * dn.to(F64)).sum(), leaves)
    for name, a, e in zip(("r", "n"), outs, (r2, n)):
        e_ = rel_l2(a, e)
        say(f"block {name}: rel-L2 {e_:.2e}")
        assert e_ <= F32_TOL
    for name, a, e in zip("q k v f gate res w b wn scale".split(), grads, want):
        e_ = rel_l2(a, e)
        say(f"block grad {name}: rel-L2 {e_:.2e}")
        assert e_ <= F32_TOL, name


def test_norms_in_a_graph_and_on_another_stream():
    """Norms forward and backward captured together: every replay, with eager calls between, equals the eager
    call bit for bit; so does a call on another stream."""
    g = torch.Generator().manual_seed(50)
    B, H, T, dv = 2, 4, 200, 128
    y, z = rnd(g, B, H, T, dv, dtype=torch.bfloat16).to(DEV), rnd(g, B, T, H, dv, dtype=torch.bfloat16).to(DEV)
    w, b, wn = rnd(g, H, dv).to(DEV), rnd(g, H, dv).to(DEV), rnd(g, H * dv).to(DEV)

    def step():
        o = ret.group_norm_gated(y, z, w, b)
        gy, gz, gw, gb = ret.group_norm_gated_bwd(y, z, o, w, b)
        flat = o.view(B, T, H * dv)
        r, n = ret.residual_norm(flat, gz.view(B, T, H * dv), wn, scale=wn)
        return (o, gy, gz, gw, gb, r, n, *(t for t in ret.residual_norm_bwd(r, n, r, wn, flat, wn, bias_grad=True)))

    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(other, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(4):
        for t in got:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want)), i
        ret.group_norm_gated_bwd(y[:, :, :77], z[:, :77], z[:, :77], w, b)
        torch.cuda.synchronize()

"""Error bounds of the attention calls against exact values, element by element.

u = 2^-24; e is what rounding a probability or a score's gradient to the tensors'
type loses (bf16: 2^-8 of it; fp32: nothing), half an output's own rounding.
A score is d products and additions: off by (d + 8) u of the sum of magnitudes,
and the exponent's argument (score times scale log2 e, less the running maximum)
by 6 u of what it is formed from.  exp2 is within 4 u.  So a probability is off
by delta_t (the row's largest such error) of itself, a softmax weight by
2 delta_t + (S + 16) u (its sum has S terms), an output by that, e and (S + 16) u
of sum A |v|.  The gradients follow their formulas term by term; every sum of n
terms adds (n + 16) u of its magnitudes.  A factor of 1.05 covers products of
two errors.
"""
import torch

import oracle

F64, U = torch.float64, 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
ROUND = {torch.float32: 0.0, torch.bfloat16: 2.0 ** -8}


def up(t):
    return None if t is None else t.detach().cpu().to(F64)


def bounds(q, k, v, lam=None, causal=True, scale=None, offset=None, lens=None, grad_o=None, few=False):
    """Errors allowed to o, lse, second and (with grad_o) grad_q, grad_k, grad_v, grad_lam, by name.
    few: no sequence has over 32 keys, so that D_m is sum A_m dP in fp32 and not from the rounded o and second."""
    dtype = q.dtype
    half, e = HALF[dtype], ROUND[dtype]
    q, k, v, lam, do = up(q), up(k), up(v), up(lam), up(grad_o)
    B, H, T, dk = q.shape
    Hk, S, dv = k.shape[1], k.shape[2], v.shape[-1]
    maps = 1 if lam is None else 2
    d = dk // maps
    scale = d ** -0.5 if scale is None else scale
    offset = S - T if offset is None else offset
    out = dict(o=torch.zeros(B, H, T, dv, dtype=F64), lse=torch.zeros(B, H, maps, T, dtype=F64),
               second=torch.zeros(B, H, T, dv, dtype=F64))
    if do is not None:
        out.update(gq=torch.zeros_like(q), gk=torch.zeros_like(k), gv=torch.zeros_like(v), gl=torch.zeros(H, dtype=F64))
        mag = {n: torch.zeros_like(out[n]) for n in ("gk", "gv")}
    o, lse, _ = oracle.attention(q, k, v, lam, causal, scale, offset, lens)
    from oracle.attention_oracle import visible
    for b in range(B):
        n = S if lens is None else min(max(int(lens[b]), 0), S)
        m = visible(T, S, n, causal, offset)
        live = torch.arange(S)[:, None] < n
        for h in range(H):
            hk = h // (H // Hk)
            kk, vv = torch.where(live, k[b, hk], 0.0), torch.where(live, v[b, hk], 0.0)
            A, dA, eo, y, w = [], [], [], [], [1.0] + ([] if lam is None else [float(lam[h])])
            for i in range(maps):
                p = slice(i * d, (i + 1) * d)
                X, aX = scale * q[b, h, :, p] @ kk[:, p].T, scale * q[b, h, :, p].abs() @ kk[:, p].abs().T
                X, aX = X.masked_fill(~m, 0), aX.masked_fill(~m, 0)
                big = X.abs().amax(-1, keepdim=True) if S else torch.zeros(T, 1, dtype=F64)
                arg = (d + 8) * U * aX + 6 * U * (X.abs() + big)
                delta = (1.01 * arg.amax(-1, keepdim=True) if S else torch.zeros(T, 1, dtype=F64)) + 4 * U
                L = lse[b, h, i][:, None]
                L = torch.where(torch.isinf(L), torch.zeros_like(L), L)
                a = torch.where(m, torch.exp(X - L), torch.zeros_like(X))
                eL = delta + (S + 16) * U + 6 * U * L.abs()
                out["lse"][b, h, i] = eL[:, 0]
                A.append(a)
                dA.append(1.01 * (arg + eL + 3 * U * L.abs()) + 4 * U)
                y.append(a @ vv)
                eo.append((2 * delta + (2 * S + 32) * U + e) * (a @ vv.abs()))
            out["o"][b, h] = eo[0] + half * o[b, h].abs() + 2 * U * y[0].abs()
            if maps > 1:
                out["o"][b, h] += abs(w[1]) * (eo[1] + 4 * U * y[1].abs())
                out["second"][b, h] = eo[1] + half * y[1].abs()
            if do is None:
                continue
            g = do[b, h]
            dP, eP = g @ vv.T, (dv + 4) * U * g.abs() @ vv.abs().T
            D, eD = [None] * maps, [None] * maps
            if maps > 1:
                D[1] = (g * y[1]).sum(-1, keepdim=True)
                eD[1] = (g.abs() * (out["second"][b, h] + (dv + 8) * U * y[1].abs())).sum(-1, keepdim=True)
            D[0] = (g * y[0]).sum(-1, keepdim=True)
            eD[0] = (g.abs() * (out["o"][b, h] + (dv + 8) * U * o[b, h].abs())).sum(-1, keepdim=True)
            if maps > 1:
                eD[0] += abs(w[1]) * (eD[1] + 4 * U * D[1].abs()) + 4 * U * D[0].abs()
            if few:
                eD = [(A[i] * (dA[i] * dP.abs() + eP + (S + 8) * U * dP.abs())).sum(-1, keepdim=True) for i in range(maps)]
            W, eW = torch.zeros_like(dP), torch.zeros_like(dP)
            for i in range(maps):
                p = slice(i * d, (i + 1) * d)
                t = (dP - D[i]).abs()
                ds = abs(w[i]) * A[i] * t
                eds = abs(w[i]) * A[i] * (dA[i] * t + eP + eD[i] + 6 * U * t) + e * ds
                out["gq"][b, h][:, p] += scale * ((eds + (S + 16) * U * ds) @ kk[:, p].abs())
                out["gk"][b, hk][:, p] += scale * (eds.T @ q[b, h, :, p].abs())
                mag["gk"][b, hk][:, p] += scale * (ds.T @ q[b, h, :, p].abs())
                W += (w[i] if i == 0 else -w[i]) * A[i]
                eW += abs(w[i]) * A[i] * (dA[i] + 4 * U)
            out["gv"][b, hk] += (eW + e * W.abs()).T @ g.abs()
            mag["gv"][b, hk] += W.abs().T @ g.abs()
            if maps > 1:
                out["gl"][h] += (A[1] * (dA[1] * dP.abs() + eP + (S + B * T + 64) * U * dP.abs())).sum()
    if do is not None:
        want = oracle.attention_backward(q, k, v, do, lam, causal, scale, offset, lens)
        for name, x in zip(("gq", "gk", "gv"), want):
            if name in mag:
                out[name] += (T * (H // Hk) + 16) * U * mag[name]
            out[name] += half * x.abs()
        if maps > 1:
            out["gl"] += 2 * U * want[3].abs()
    return {n: 1.05 * x for n, x in out.items()}


def close(name, got, want, bound):
    """|got - want| <= bound, element by element; infinities have to agree."""
    got, want = up(got), up(want)
    assert got.shape == want.shape, (name, got.shape, want.shape)
    fine = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), fine) and torch.equal(got[~fine], want[~fine]), name
    over = ((got - want).abs()[fine] / (bound[fine] + 1e-37))
    worst = float(over.max()) if over.numel() else 0.0
    print(f"{name}: worst error {worst:.3f} of its bound", flush=True)
    assert worst <= 1.0, (name, worst)

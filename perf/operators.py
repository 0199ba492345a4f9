"""Cases, plain forms and 64-bit values of the gated-block operators.

Three operators around a recurrent token mixer, each with its gradient:

  scan           gated linear recurrence h_t = a_t h_(t-1) + u_t with a_t = sigmoid(f_t)^rate and
                 u_t = x_t or (1 - a_t) x_t; its single-token step; its backward pass
  gate_norm      per-head GroupNorm of a mixer's output, times silu(gate), written with the heads merged
  residual_norm  r = alpha x + scale f and n = norm(r): the residual stream after a block and the
                 next block's normalised input

`own` chooses between the plain forms (elementary torch operations in 32 bits) and the library's calls.
Shapes are those of the library's workloads (8 or 16 heads with values of 512, widths of 2048 and 4096,
2048, 8192 and 65536 tokens, 128 decode streams) and generic odd ones.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-5


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token for each of 8 streams: the latency of a call
        dict(name="scan_step", op="scan", do="step", B=8, H=8, T=1, d=512, dtype="bf16", normalize=True, state=True, reset=0.0),
        # a prompt of 4 x 2048 tokens, continued from no state
        dict(name="scan_prompt", op="scan", do="fwd", B=4, H=8, T=2048, d=512, dtype="bf16", normalize=True, state=False, reset=0.0),
        # one long context of 65536 tokens in packed documents (a gate of -inf starts each), carried state
        dict(name="scan_long", op="scan", do="fwd", B=1, H=8, T=65536, d=512, dtype="bf16", normalize=False, state=True, reset=1 / 2048),
        # a training step's forward and backward on 2 x 8192 tokens
        dict(name="scan_train", op="scan", do="train", B=2, H=16, T=8192, d=512, dtype="bf16", normalize=True, state=False, reset=0.0),
        # odd sizes in 32 bits, forward and backward with a carried state and its gradient
        dict(name="scan_train_odd", op="scan", do="train", B=3, H=5, T=1337, d=201, dtype="f32", normalize=False, state=True, reset=1 / 300),
        # the output of a decode step of 128 streams
        dict(name="gate_norm_decode", op="gate_norm", do="fwd", B=128, H=16, T=1, d=512, dtype="bf16", affine=True),
        # the output of the long context
        dict(name="gate_norm_long", op="gate_norm", do="fwd", B=1, H=8, T=65536, d=512, dtype="bf16", affine=True),
        # the backward pass of a 4 x 2048 training step
        dict(name="gate_norm_train", op="gate_norm", do="bwd", B=4, H=8, T=2048, d=512, dtype="bf16", affine=True),
        # the backward pass at odd sizes in 32 bits
        dict(name="gate_norm_odd", op="gate_norm", do="bwd", B=3, H=5, T=777, d=101, dtype="f32", affine=True),
        # a decode step of 128 streams, width 2048, LayerNorm
        dict(name="residual_norm_decode", op="residual_norm", do="fwd", rows=128, D=2048, dtype="bf16", rms=False, affine=True, scale=False, alpha=1.0),
        # a prompt at an odd width in 32 bits, RMSNorm, a channel scale and a weighted residual
        dict(name="residual_norm_odd", op="residual_norm", do="fwd", rows=8191, D=1111, dtype="f32", rms=True, affine=True, scale=True, alpha=1.5),
        # the backward pass of 2 x 8192 tokens, width 4096, LayerNorm with a channel scale
        dict(name="residual_norm_train", op="residual_norm", do="bwd", rows=16384, D=4096, dtype="bf16", rms=False, affine=True, scale=True, alpha=1.0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scan", "gate_norm", "residual_norm"])
    dtype = rng.choice(["bf16", "f32"])
    most = 1 << 26  # elements: below the largest listed case in either type
    if op == "residual_norm":
        D = _log(rng, 16, 8192)
        return dict(op=op, do=rng.choice(["fwd", "bwd"]), rows=_log(rng, 1, min(65536, most // D)), D=D, dtype=dtype,
                    rms=rng.random() < 0.5, affine=rng.random() < 0.8, scale=rng.random() < 0.5, alpha=rng.choice([1.0, 0.5, 1.7]))
    B, H, d = _log(rng, 1, 32), rng.randint(1, 16), _log(rng, 8, 512)
    if rng.random() < 0.4:
        d = -(-d // 8) * 8
    T = _log(rng, 1, max(1, min(65536, most // (B * H * d))))
    if op == "gate_norm":
        return dict(op=op, do=rng.choice(["fwd", "bwd"]), B=B, H=H, T=T, d=d, dtype=dtype, affine=rng.random() < 0.8)
    do = rng.choice(["fwd", "train", "train", "step"])
    return dict(op=op, do=do, B=B, H=H, T=1 if do == "step" else T, d=d, dtype=dtype, normalize=rng.random() < 0.5,
                state=do == "step" or rng.random() < 0.6, reset=rng.choice([0.0, 1 / 64, 1 / 1024]))


def _rates(H):
    """Decay exponents of the heads, 1 down to 1/16: short to long memories, as multi-scale decays have."""
    return [2.0 ** (-4.0 * h / max(1, H - 1)) for h in range(H)]


def _inputs(c, seed, dev):
    """Every tensor of a case, by name, from the seed alone."""
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[c["dtype"]]

    def normal(*shape, dtype=dt, scale=1.0, shift=0.0):
        return torch.randn(shape, generator=g, device=dev).mul_(scale).add_(shift).to(dtype)

    f32 = torch.float32
    s = {}
    if c["op"] == "scan":
        B, H, T, d = c["B"], c["H"], c["T"], c["d"]
        shape = (B, H, d) if c["do"] == "step" else (B, H, T, d)
        s["x"] = normal(*shape)
        s["f"] = normal(*shape, scale=1.5, shift=2.0)  # gates of a trained layer lean towards remembering
        if c["reset"] and c["do"] != "step":  # first tokens of packed documents forget everything before them
            first = torch.rand((B, 1, T, 1), generator=g, device=dev) < c["reset"]
            s["f"].masked_fill_(first, -math.inf)
        if c["state"]:
            s["state"] = normal(B, H, d, dtype=f32)
        if c["do"] == "train":
            s["dy"] = normal(*shape)
            if c["state"]:
                s["dstate"] = normal(B, H, d, dtype=f32)
    elif c["op"] == "gate_norm":
        B, H, T, d = c["B"], c["H"], c["T"], c["d"]
        s["y"] = normal(B, H, T, d, scale=0.3, shift=0.05)
        s["gate"] = normal(B, T, H, d)
        if c["affine"]:
            s["weight"], s["bias"] = normal(H, d, dtype=f32, scale=0.2, shift=1.0), normal(H, d, dtype=f32, scale=0.1)
        if c["do"] == "bwd":
            s["dout"] = normal(B, T, H, d)
    else:
        R, D = c["rows"], c["D"]
        if c["do"] == "fwd":
            s["x"], s["f"] = normal(R, D, scale=2.0), normal(R, D)
        else:
            s["r"], s["dn"], s["dr"] = normal(R, D, scale=2.0), normal(R, D), normal(R, D)
            if c["scale"]:
                s["f"] = normal(R, D)
        if c["affine"]:
            s["weight"] = normal(D, dtype=f32, scale=0.2, shift=1.0)
            if not c["rms"]:
                s["bias"] = normal(D, dtype=f32, scale=0.1)
        if c["scale"]:
            s["scale"] = normal(D, dtype=f32, scale=0.1, shift=0.5)
    return s


def prepare(case, seed):
    s = _inputs(case, seed, "cuda")
    s["case"] = case
    if case["op"] == "scan":
        s["rates"] = _rates(case["H"])  # a host list, as the library's per-head decays are
    return s


# ------------------------------------------------------------------ plain forms
def _gate(f, rates):
    """log a, a and 1 - a of a_t = sigmoid(f_t)^rate."""
    rate = torch.tensor(rates, device=f.device, dtype=f.dtype).view(1, -1, *([1] * (f.dim() - 2)))
    z = -rate * (torch.clamp(-f, min=0) + torch.log1p(torch.exp(-f.abs())))
    return torch.exp(z), -torch.expm1(z), rate


def _scan(a, u):
    """h_t = a_t h_(t-1) + u_t along dim 2 from h = 0: neighbours are joined, the half as long scan gives every
    second value, and one more step gives the others."""
    T = u.shape[2]
    if T == 1:
        return u
    n = T // 2
    a0, a1, u0, u1 = a[:, :, 0 : 2 * n : 2], a[:, :, 1::2], u[:, :, 0 : 2 * n : 2], u[:, :, 1::2]
    h = torch.empty_like(u)
    odd = _scan(a0 * a1, torch.addcmul(u1, a1, u0))
    h[:, :, 1::2] = odd
    h[:, :, 0] = u[:, :, 0]
    if T > 2:
        h[:, :, 2::2] = torch.addcmul(u[:, :, 2::2], a[:, :, 2::2], odd[:, :, : (T - 1) // 2])
    return h


def _plain_scan(s):
    c = s["case"]
    x, f = s["x"].float(), s["f"].float()
    dt = s["x"].dtype
    a, na, rate = _gate(f, s["rates"])
    u = na * x if c["normalize"] else x.clone()
    if c["do"] == "step":
        s["state"].copy_(torch.addcmul(u, a, s["state"]))
        return {"y": s["state"].to(dt), "state": s["state"]}
    state = s.get("state")
    if state is not None:
        u[:, :, 0] += a[:, :, 0] * state
    h = _scan(a, u)
    out = {"y": h.to(dt), "state": h[:, :, -1].contiguous()}
    if c["do"] == "fwd":
        return out
    g = s["dy"].float()
    if state is not None:
        g[:, :, -1] += s["dstate"]
    later = torch.cat([a[:, :, 1:], torch.zeros_like(a[:, :, :1])], dim=2)  # a_(t+1)
    g = _scan(later.flip(2), g.flip(2)).flip(2)  # dL/dh_t
    before = torch.cat([(torch.zeros_like(h[:, :, 0]) if state is None else state).unsqueeze(2), h[:, :, :-1]], dim=2)
    da = g * (before - x) if c["normalize"] else g * before
    out["dx"] = (g * na if c["normalize"] else g).to(dt)
    out["df"] = (da * a * rate * torch.sigmoid(-f)).to(dt)
    if state is not None:
        out["dstate"] = (a[:, :, 0] * g[:, :, 0])
    return out


def _own_scan(s):
    import retnet_retention_chunkwise_amd as ret

    c = s["case"]
    if c["do"] == "step":
        y = ret.gated_scan_step(s["x"], s["f"], s["rates"], s["state"], normalize=c["normalize"])
        return {"y": y, "state": s["state"]}
    state = s.get("state")
    if c["do"] == "fwd":
        y, last = ret.gated_scan_fwd(s["x"], s["f"], s["rates"], state_in=state, normalize=c["normalize"])
        return {"y": y, "state": last}
    y, last, kept = ret.gated_scan_fwd(s["x"], s["f"], s["rates"], state_in=state, normalize=c["normalize"], checkpoints=True)
    dx, df, ds = ret.gated_scan_bwd(s["x"], s["f"], s["rates"], s["dy"], state_in=state, grad_state_out=s.get("dstate"),
                                    checkpoints=kept, normalize=c["normalize"], grad_state_in=state is not None)
    out = {"y": y, "state": last, "dx": dx, "df": df}
    if state is not None:
        out["dstate"] = ds
        if s["dy"].dtype == torch.float32:
            # float() is no copy in 32 bits, so the plain pass leaves the state's gradient added to the last
            # token's dy: a second pass on the same state starts from that, here as there
            s["dy"][:, :, -1] += s["dstate"]
    return out


def _plain_gate_norm(s):
    c = s["case"]
    dt = s["y"].dtype
    y, z = s["y"].float(), s["gate"].float()
    mu = y.mean(-1, keepdim=True)
    rstd = torch.rsqrt((y - mu).square().mean(-1, keepdim=True) + EPS)
    xh = (y - mu) * rstd
    w, b = s.get("weight"), s.get("bias")
    n = xh if w is None else xh * w[:, None] + b[:, None]
    sig = torch.sigmoid(z)
    if c["do"] == "fwd":
        return {"out": (n.transpose(1, 2) * (z * sig)).to(dt)}
    do = s["dout"].float()
    dz = do * n.transpose(1, 2) * (sig * (1 + z * (1 - sig)))
    dn = (do * (z * sig)).transpose(1, 2)
    dh = dn if w is None else dn * w[:, None]
    dy = rstd * (dh - dh.mean(-1, keepdim=True) - xh * (dh * xh).mean(-1, keepdim=True))
    out = {"dy": dy.to(dt), "dgate": dz.to(dt)}
    if w is not None:
        out["dweight"], out["dbias"] = (dn * xh).sum((0, 2)), dn.sum((0, 2))
    return out


def _own_gate_norm(s):
    import retnet_retention_chunkwise_amd as ret

    w, b = s.get("weight"), s.get("bias")
    if s["case"]["do"] == "fwd":
        return {"out": ret.group_norm_gated(s["y"], s["gate"], w, b, EPS)}
    dy, dz, dw, db = ret.group_norm_gated_bwd(s["y"], s["gate"], s["dout"], w, b, EPS)
    out = {"dy": dy, "dgate": dz}
    if w is not None:
        out["dweight"], out["dbias"] = dw, db
    return out


def _plain_residual_norm(s):
    c = s["case"]
    w, b, scale = s.get("weight"), s.get("bias"), s.get("scale")
    if c["do"] == "fwd":
        dt = s["x"].dtype
        f = s["f"].float()
        r = (c["alpha"] * s["x"].float() + (f if scale is None else f * scale)).to(dt)  # the stream is held in its type
        h = r.float()
        if not c["rms"]:
            h = h - h.mean(-1, keepdim=True)
        n = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS)
        n = n if w is None else n * w
        n = n if b is None else n + b
        return {"r": r, "n": n.to(dt)}
    dt = s["r"].dtype
    h, dn = s["r"].float(), s["dn"].float()
    if not c["rms"]:
        h = h - h.mean(-1, keepdim=True)
    rstd = torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS)
    xh = h * rstd
    dh = dn if w is None else dn * w
    g = dh - xh * (dh * xh).mean(-1, keepdim=True)
    if not c["rms"]:
        g = g - dh.mean(-1, keepdim=True)
    g = s["dr"].float() + rstd * g
    out = {"dx": (c["alpha"] * g).to(dt), "df": (g if scale is None else g * scale).to(dt)}
    if w is not None:
        out["dweight"] = (dn * xh).sum(0)
        if b is not None:
            out["dbias"] = dn.sum(0)
    if scale is not None:
        out["dscale"] = (g * s["f"].float()).sum(0)
    return out


def _own_residual_norm(s):
    import retnet_retention_chunkwise_amd as ret

    c = s["case"]
    w, b, scale = s.get("weight"), s.get("bias"), s.get("scale")
    if c["do"] == "fwd":
        r, n = ret.residual_norm(s["x"], s["f"], w, b, scale=scale, alpha=c["alpha"], eps=EPS, rms=c["rms"])
        return {"r": r, "n": n}
    dx, df, dw, db, dscale = ret.residual_norm_bwd(s["r"], s["dn"], s["dr"], w, f=s.get("f"), scale=scale, alpha=c["alpha"],
                                                   eps=EPS, rms=c["rms"], bias_grad=b is not None)
    out = {"dx": dx, "df": df}
    if w is not None:
        out["dweight"] = dw
        if b is not None:
            out["dbias"] = db
    if scale is not None:
        out["dscale"] = dscale
    return out


def run(state):
    op = state["case"]["op"]
    if own:
        return {"scan": _own_scan, "gate_norm": _own_gate_norm, "residual_norm": _own_residual_norm}[op](state)
    return {"scan": _plain_scan, "gate_norm": _plain_gate_norm, "residual_norm": _plain_residual_norm}[op](state)


def work(case):
    """Bytes of inputs and outputs, each moved once, and the operations of the formulas (a transcendental counts as one)."""
    c, e = case, 2 if case["dtype"] == "bf16" else 4
    if c["op"] == "scan":
        vec = c["B"] * c["H"] * c["d"]
        n = vec * c["T"]
        states = 4 * vec * (1 + c["state"])
        if c["do"] == "train":  # x, f, dy in; y, dx, df out
            return {"bytes": 6 * n * e + states + 8 * vec * c["state"], "flops": 32 * n}
        return {"bytes": 3 * n * e + states, "flops": 12 * n}
    if c["op"] == "gate_norm":
        n = c["B"] * c["H"] * c["T"] * c["d"]
        vec = 8 * c["H"] * c["d"] if c["affine"] else 0
        return {"bytes": 3 * n * e + vec, "flops": 14 * n} if c["do"] == "fwd" else {"bytes": 5 * n * e + 2 * vec, "flops": 34 * n}
    n, D = c["rows"] * c["D"], c["D"]
    vecs = (c["affine"] * (1 if c["rms"] else 2) + c["scale"]) * D * 4
    if c["do"] == "fwd":
        return {"bytes": 4 * n * e + vecs, "flops": 10 * n}
    return {"bytes": (5 + c["scale"]) * n * e + 2 * vecs, "flops": 20 * n}


# ------------------------------------------------------------------ 64 bits, from the definitions
def exact(case, seed):
    s = _inputs(case, seed, "cuda")
    held = s["r" if "r" in s else "y" if "y" in s else "x"].dtype
    s = {k: v.double() for k, v in s.items()}
    with torch.no_grad():
        return {"scan": _exact_scan, "gate_norm": _exact_gate_norm, "residual_norm": _exact_residual_norm}[case["op"]](case, s, held)


def _exact_scan(c, s, held):
    B, H, d = c["B"], c["H"], c["d"]
    one = c["do"] == "step"
    steps = lambda t: (t.unsqueeze(2) if one else t).permute(2, 0, 1, 3).contiguous()  # noqa: E731  [T,B,H,d]
    x, f = steps(s["x"]), steps(s["f"])
    T = x.shape[0]
    rate = torch.tensor(_rates(H), dtype=torch.float64, device=x.device).view(1, 1, H, 1)
    loga = rate * torch.nn.functional.logsigmoid(f)
    a = torch.exp(loga)
    u = -torch.expm1(loga) * x if c["normalize"] else x
    h = s["state"] if c["state"] else torch.zeros(B, H, d, dtype=torch.float64, device=x.device)
    all_h = torch.empty(T + 1, B, H, d, dtype=torch.float64, device=x.device)
    all_h[0] = h
    for t in range(T):
        torch.addcmul(u[t], a[t], all_h[t], out=all_h[t + 1])
    back = lambda t: t.permute(1, 2, 0, 3).contiguous()  # noqa: E731
    if one:
        return {"y": all_h[1], "state": all_h[1]}
    out = {"y": back(all_h[1:]), "state": all_h[T].clone()}
    if c["do"] == "fwd":
        return out
    g = steps(s["dy"])
    if c["state"]:
        g[T - 1] += s["dstate"]
    for t in range(T - 1, 0, -1):
        g[t - 1].addcmul_(a[t], g[t])
    prev = all_h[:T]
    keep = torch.sigmoid(-f)  # d softplus(-f) / d(-f)
    out["dx"] = back(g * -torch.expm1(loga) if c["normalize"] else g)
    out["df"] = back(g * ((prev - x) if c["normalize"] else prev) * a * rate * keep)
    if c["state"]:
        out["dstate"] = a[0] * g[0]
    return out


def _exact_gate_norm(c, s, held):
    y, z = s["y"], s["gate"].permute(0, 2, 1, 3)  # gate as [B,H,T,d]
    one = torch.ones(c["H"], c["d"], dtype=torch.float64, device=y.device)
    w, b = (s["weight"], s["bias"]) if c["affine"] else (one, 0 * one)
    w, b = w[None, :, None], b[None, :, None]
    var, mu = torch.var_mean(y, dim=-1, correction=0, keepdim=True)
    sd = torch.sqrt(var + EPS)
    hat = (y - mu) / sd
    n, swish, sg = hat * w + b, z / (1 + torch.exp(-z)), 1 / (1 + torch.exp(-z))
    merge = lambda t: t.permute(0, 2, 1, 3).contiguous()  # noqa: E731
    if c["do"] == "fwd":
        return {"out": merge(n * swish)}
    do = s["dout"].permute(0, 2, 1, 3)
    dn = do * swish
    p = dn * w
    out = {"dy": (p - p.mean(-1, keepdim=True) - hat * (p * hat).mean(-1, keepdim=True)) / sd,
           "dgate": merge(do * n * (sg + swish * (1 - sg)))}
    if c["affine"]:
        out["dweight"], out["dbias"] = (dn * hat).sum(dim=(0, 2)), dn.sum(dim=(0, 2))
    return out


def _exact_residual_norm(c, s, held):
    dev = s["x" if c["do"] == "fwd" else "r"].device
    one = torch.ones(c["D"], dtype=torch.float64, device=dev)
    w, b, g = s.get("weight", one), s.get("bias", 0 * one), s.get("scale", one)
    r = c["alpha"] * s["x"] + g * s["f"] if c["do"] == "fwd" else s["r"]
    m = r.float().to(held).double() if c["do"] == "fwd" else r  # the norm sees the stream as it is held
    mu = torch.zeros_like(m[:, :1]) if c["rms"] else m.mean(-1, keepdim=True)
    sd = torch.sqrt((m - mu).square().mean(-1, keepdim=True) + EPS)
    hat = (m - mu) / sd
    if c["do"] == "fwd":
        return {"r": r, "n": hat * w + b}
    p = s["dn"] * w
    t = p - hat * (p * hat).mean(-1, keepdim=True)
    if not c["rms"]:
        t = t - p.mean(-1, keepdim=True)
    t = s["dr"] + t / sd
    out = {"dx": c["alpha"] * t, "df": g * t}
    if c["affine"]:
        out["dweight"] = (s["dn"] * hat).sum(0)
        if not c["rms"]:
            out["dbias"] = s["dn"].sum(0)
    if c["scale"]:
        out["dscale"] = (t * s["f"]).sum(0)
    return out

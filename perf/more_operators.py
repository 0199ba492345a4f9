"""Cases, plain forms and 64-bit values of the attention operators.

Softmax attention beside retention in a hybrid stack, ordinary (one map) or differential (the difference of
two maps, the second with a learned weight per head), query heads sharing key and value heads:

  attn    a whole sequence: forward, or a training step's forward and backward
  step    one new token of each sequence over a paged cache of keys and values, into which it is stored
  append  the keys and values of a prompt into the pages of the cache

`own` chooses between the plain forms (elementary torch operations in 32 bits) and the library's calls.
Shapes are those of the library's workloads (8 or 16 heads with keys of 256, 2048 and 8192 tokens, 128 decode
streams, 65536 tokens) and generic odd ones.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # a prompt of 4 x 2048 tokens, wide heads
        dict(name="attn_prompt", op="attn", do="fwd", B=4, H=8, Hk=8, T=2048, S=2048, dk=256, dv=256, dtype="bf16", diff=True, causal=True, ragged=False),
        # a long prompt, four query heads to a key head
        dict(name="attn_long", op="attn", do="fwd", B=1, H=16, Hk=4, T=8192, S=8192, dk=128, dv=128, dtype="bf16", diff=True, causal=True, ragged=False),
        # a few new tokens over a long context that is already there (continuation, checked drafts)
        dict(name="attn_continue", op="attn", do="fwd", B=2, H=8, Hk=2, T=16, S=8192, dk=128, dv=128, dtype="bf16", diff=True, causal=True, ragged=False),
        # a training step's forward and backward on 2 x 4096 tokens
        dict(name="attn_train", op="attn", do="train", B=2, H=16, Hk=4, T=4096, S=4096, dk=128, dv=128, dtype="bf16", diff=True, causal=True, ragged=False),
        # an encoder's training step: ordinary softmax, both directions, a padded batch of odd length
        dict(name="attn_train_padded", op="attn", do="train", B=6, H=12, Hk=12, T=777, S=777, dk=64, dv=64, dtype="bf16", diff=False, causal=False, ragged=True),
        # odd sizes in 32 bits, padded, shared key heads
        dict(name="attn_train_odd", op="attn", do="train", B=3, H=6, Hk=2, T=501, S=501, dk=80, dv=72, dtype="f32", diff=True, causal=True, ragged=True),
        # one token for each of 8 streams over short contexts: the latency of a call
        dict(name="step_small", op="step", B=8, H=8, Hk=8, S=512, page=64, dk=128, dv=128, dtype="bf16", diff=True, ragged=False),
        # a decode step of 128 streams
        dict(name="step_batch", op="step", B=128, H=16, Hk=4, S=2048, page=64, dk=128, dv=128, dtype="bf16", diff=True, ragged=True),
        # two streams over 65536 tokens each in small pages, ordinary softmax
        dict(name="step_long", op="step", B=2, H=32, Hk=8, S=65536, page=16, dk=128, dv=128, dtype="bf16", diff=False, ragged=False),
        # odd sizes in 32 bits, pages that end inside any tile, streams from empty to full
        dict(name="step_odd", op="step", B=5, H=6, Hk=3, S=3001, page=24, dk=72, dv=80, dtype="f32", diff=True, ragged=True),
        # the prompts of attn_prompt into the cache
        dict(name="append_prompt", op="append", B=4, Hk=8, T=2048, S=4096, page=64, dk=256, dv=256, dtype="bf16", ragged=False),
        # a few accepted tokens of each of 128 streams, another number for each
        dict(name="append_few", op="append", B=128, Hk=4, T=5, S=2048, page=16, dk=128, dv=128, dtype="bf16", ragged=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "step", "step", "append"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    Hk, diff = rng.randint(1, 8), rng.random() < 0.6
    H = Hk * rng.choice([1, 1, 2, 3, 4, 8])
    # channels: multiples of 8 mostly, as models have them, any number sometimes
    dk = 2 * _log(rng, 8, 128) if diff else _log(rng, 16, 256)
    dv = _log(rng, 16, 256)
    if rng.random() < 0.7:
        dk, dv = -(-dk // 16) * 16, -(-dv // 8) * 8
    B = _log(rng, 1, 16)
    if op == "attn":
        do = rng.choice(["fwd", "train"])
        most = 1 << (28 if dtype == "bf16" else 26)  # pairs, of heads up to twice as wide as the largest listed case's
        if do == "fwd" and rng.random() < 0.4:  # new tokens over a context
            T = _log(rng, 1, 300)
            S = T + _log(rng, 1, max(2, min(16384, (1 << 26) // (B * H * T))))
        else:
            # one token alone has no gradient at its score: training starts at two
            T = S = _log(rng, 2 if do == "train" else 1, max(16, min(4096, int(math.sqrt(most / (B * H))))))
        return dict(op=op, do=do, B=B, H=H, Hk=Hk, T=T, S=S, dk=dk, dv=dv, dtype=dtype, diff=diff, causal=T != S or rng.random() < 0.7,
                    ragged=B > 1 and T == S and rng.random() < 0.4)
    page = rng.choice([1, 16, 16, 24, 64, 64, 100, 256])
    if op == "step":
        B = _log(rng, 1, 256)
        S = _log(rng, 1, max(16, min(65536, (1 << 26) // (B * Hk * (dk + dv)))))
        return dict(op=op, B=B, H=H, Hk=Hk, S=S, page=page, dk=dk, dv=dv, dtype=dtype, diff=diff, ragged=B > 1 and rng.random() < 0.6)
    T = _log(rng, 1, max(2, min(8192, (1 << 24) // (B * Hk * (dk + dv)))))
    return dict(op=op, B=B, Hk=Hk, T=T, S=T + rng.randint(0, 2000), page=page, dk=dk, dv=dv, dtype=dtype, ragged=B > 1 and rng.random() < 0.6)


def _lens(c):
    """Keys of each sequence (attn), tokens cached before the call (step, append), tokens to store (append)."""
    B, S = c["B"], c["S"]
    if c["op"] == "attn":
        return [S - S * b // B for b in range(B)] if c["ragged"] else [S] * B
    if c["op"] == "step":
        return [(S - 1) * b // (B - 1) for b in range(B)] if c["ragged"] else [S - 1] * B
    return [(S - c["T"]) * b // max(1, B - 1) for b in range(B)]


def _counts(c):
    return [1 + (b * 7) % c["T"] for b in range(c["B"])] if c["ragged"] else [c["T"]] * c["B"]


def _pages(c):
    return -(-c["S"] // c["page"])


def _inputs(c, seed, dev):
    """Every tensor of a case, by name, from the seed alone."""
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[c["dtype"]]

    def normal(*shape, dtype=dt, scale=1.0, shift=0.0):
        return torch.randn(shape, generator=g, device=dev).mul_(scale).add_(shift).to(dtype)

    i32 = dict(dtype=torch.int32, device=dev)
    B, Hk, S, dk, dv = c["B"], c["Hk"], c["S"], c["dk"], c["dv"]
    s = {}
    if c["op"] == "attn":
        # scores of unit scale and a half: rows of a trained layer look at some of their keys
        s["q"], s["k"], s["v"] = normal(B, c["H"], c["T"], dk, scale=1.5), normal(B, Hk, S, dk), normal(B, Hk, S, dv)
        if c["ragged"]:
            s["lens"] = torch.tensor(_lens(c), **i32)
        if c["do"] == "train":
            s["do"] = normal(B, c["H"], c["T"], dv)
            if c["ragged"]:  # no loss on padding
                s["do"].masked_fill_(torch.arange(c["T"], device=dev)[None, None, :, None] >= s["lens"][:, None, None, None], 0)
    else:
        n, T = _pages(c), c.get("T", 1)
        P = B * n + 3
        s["k_cache"], s["v_cache"] = normal(P, Hk, c["page"], dk), normal(P, Hk, c["page"], dv)
        s["table"] = torch.randperm(P, generator=g, device=dev)[: B * n].view(B, n).to(torch.int32)
        s["lens"] = torch.tensor(_lens(c), **i32)
        if c["op"] == "step":
            s["q"], s["k"], s["v"] = normal(B, c["H"], dk, scale=1.5), normal(B, Hk, dk), normal(B, Hk, dv)
        else:
            s["k"], s["v"] = normal(B, Hk, T, dk), normal(B, Hk, T, dv)
            s["counts"] = torch.tensor(_counts(c), **i32)
    if c.get("diff"):
        s["lam"] = normal(c["H"], dtype=torch.float32, scale=0.15, shift=0.6)
    return s


def prepare(case, seed):
    s = _inputs(case, seed, "cuda")
    s["case"] = case
    return s


# ------------------------------------------------------------------ plain forms
def _maps(q, k, diff):
    """q [..,R,dk], k [..,S,dk] as maps [..,M,R,d], [..,M,S,d]."""
    M = 2 if diff else 1
    return q.unflatten(-1, (M, -1)).transpose(-2, -3), k.unflatten(-1, (M, -1)).transpose(-2, -3)


def _softmax(x, seen):
    """Softmax of x over the seen keys; rows that see none are zero."""
    x = x.masked_fill(~seen, -math.inf)
    e = torch.exp(x - x.amax(-1, keepdim=True).clamp_min(torch.finfo(x.dtype).min))
    return e / e.sum(-1, keepdim=True).clamp_min(torch.finfo(x.dtype).tiny)


def _plain_attn(s):
    c = s["case"]
    dt, diff, B, H, Hk, T, S = s["q"].dtype, c["diff"], c["B"], c["H"], c["Hk"], c["T"], c["S"]
    d = c["dk"] // (2 if diff else 1)
    scale = d ** -0.5
    q, k = _maps(s["q"].float().view(B, Hk, H // Hk, T, -1), s["k"].float()[:, :, None], diff)  # [B,Hk,G,M,T,d], [B,Hk,1,M,S,d]
    v = s["v"].float()[:, :, None]  # [B,Hk,1,S,dv]
    at = torch.arange(S, device=v.device)
    seen = at < (s["lens"].view(B, 1, 1, 1, 1, 1) if "lens" in s else S)
    if c["causal"]:
        seen = seen & (at <= torch.arange(T, device=v.device)[:, None] + (S - T))
    A = _softmax(scale * (q @ k.transpose(-1, -2)), seen)  # [B,Hk,G,M,T,S]
    lam = s["lam"].view(Hk, -1, 1, 1) if diff else None
    W = A[..., 0, :, :] - lam * A[..., 1, :, :] if diff else A[..., 0, :, :]
    out = {"o": (W @ v).reshape(B, H, T, -1).to(dt)}
    if c["do"] == "fwd":
        return out
    do = s["do"].float().view(B, Hk, H // Hk, T, -1)
    out["dv"] = (W.transpose(-1, -2) @ do).sum(2).to(dt)
    dA = (do @ v.transpose(-1, -2))[..., None, :, :]  # of either map, before its weight
    dx = A * (dA - (A * dA).sum(-1, keepdim=True))
    if diff:
        out["dlam"] = -(A[..., 1, :, :] * dA[..., 0, :, :]).sum((-1, -2)).sum(0).view(H)
        dx[..., 1, :, :] *= -lam
    out["dq"] = (scale * (dx @ k)).transpose(-2, -3).reshape(B, H, T, -1).to(dt)
    out["dk"] = (scale * (dx.transpose(-1, -2) @ q).sum(2)).transpose(-2, -3).reshape(B, Hk, S, -1).to(dt)
    return out


def _own_attn(s):
    import retnet_retention_chunkwise_amd as ret

    c = s["case"]
    lam, lens = s.get("lam"), s.get("lens")
    if c["do"] == "fwd":
        return {"o": ret.attention_fwd(s["q"], s["k"], s["v"], lam, causal=c["causal"], lens=lens)}
    o, kept = ret.attention_fwd(s["q"], s["k"], s["v"], lam, causal=c["causal"], lens=lens, keep=True)
    dq, dk, dv, dlam = ret.attention_bwd(s["q"], s["k"], s["v"], o, s["do"], kept, lam, causal=c["causal"], lens=lens)
    out = {"o": o, "dv": dv}
    if lam is not None:
        out["dlam"] = dlam
    return {**out, "dq": dq, "dk": dk}


def _slots(s, at):
    """Pages and rows in them of the positions at [B,n]."""
    page = s["case"]["page"]
    return s["table"].long().gather(1, at // page), at % page


def _plain_store(s, at, k, v, stored):
    """Rows k, v [B,n,Hk,..] into the cache at the positions at [B,n] where stored."""
    p, r = _slots(s, at)
    for cache, new in ((s["k_cache"], k), (s["v_cache"], v)):
        cache[p, :, r] = torch.where(stored[..., None, None], new, cache[p, :, r])


def _plain_step(s):
    c = s["case"]
    dt, diff, B, H, Hk, S = s["q"].dtype, c["diff"], c["B"], c["H"], c["Hk"], c["S"]
    lens = s["lens"].long()
    _plain_store(s, lens[:, None], s["k"][:, None], s["v"][:, None], torch.ones_like(lens, dtype=torch.bool)[:, None])
    t = s["table"].long()
    k, v = (x[t].transpose(1, 2).flatten(2, 3).float() for x in (s["k_cache"], s["v_cache"]))  # [B,Hk,keys,..]
    q, k = _maps(s["q"].float().view(B, Hk, H // Hk, -1), k, diff)  # [B,Hk,M,G,d], [B,Hk,M,keys,d]
    scale = q.shape[-1] ** -0.5
    seen = torch.arange(k.shape[-2], device=k.device) <= lens.view(B, 1, 1, 1, 1)
    A = _softmax(scale * (q @ k.transpose(-1, -2)), seen)  # [B,Hk,M,G,keys]
    W = A[:, :, 0] - s["lam"].view(Hk, -1, 1) * A[:, :, 1] if diff else A[:, :, 0]
    o = W @ v.masked_fill(~seen[:, 0, 0, 0, :, None].unsqueeze(1), 0)
    return {"o": o.reshape(B, H, -1).to(dt), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_step(s):
    import retnet_retention_chunkwise_amd as ret

    o = ret.attention_step(s["q"], s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s.get("lam"))
    return {"o": o, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_append(s):
    t = torch.arange(s["case"]["T"], device=s["k"].device)
    at = s["lens"].long()[:, None] + t
    _plain_store(s, at, s["k"].transpose(1, 2), s["v"].transpose(1, 2), t < s["counts"][:, None])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_append(s):
    import retnet_retention_chunkwise_amd as ret

    ret.cache_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["table"], s["lens"], s["counts"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"attn": _own_attn, "step": _own_step, "append": _own_append}[op](state)
    return {"attn": _plain_attn, "step": _plain_step, "append": _plain_append}[op](state)


def work(case):
    """Bytes of inputs and outputs, each moved once, and the operations of the products over the visible pairs."""
    c, e = case, 2 if case["dtype"] == "bf16" else 4
    B, Hk, T, S, dk, dv = c["B"], c["Hk"], c.get("T", 1), c["S"], c["dk"], c["dv"]
    if c["op"] == "append":
        return {"bytes": 2 * e * Hk * (dk + dv) * sum(_counts(c)) + 4 * B * (_pages(c) + 2), "flops": 0}
    M, H, lens = 2 if c["diff"] else 1, c["H"], _lens(c)
    if c["op"] == "step":
        keys = sum(n + 1 for n in lens)
        return {"bytes": e * (Hk * (dk + dv) * (keys + B) + B * H * (dk + dv)) + 4 * B * (_pages(c) + 1), "flops": H * keys * 2 * (dk + M * dv)}
    kept = sum(lens) if c["ragged"] else B * S
    rows, keys = B * H * T * (dk + dv) * e, Hk * kept * (dk + dv) * e  # q and o; the keys and values that count
    pairs = sum(_visible(T, n, S - T) if c["causal"] else T * n for n in lens) * H
    if c["do"] == "fwd":
        return {"bytes": rows + keys, "flops": pairs * 2 * (dk + M * dv)}
    return {"bytes": 2 * rows + B * H * T * dv * e + keys + B * Hk * S * (dk + dv) * e, "flops": pairs * (2 * (dk + M * dv) + 6 * dk + 4 * dv)}


def _visible(T, n, offset):
    """Pairs s <= t + offset, s < n, of T rows."""
    ramp = max(0, min(T, n - offset))  # rows before the keys end
    return (1 + 2 * offset + ramp) * ramp // 2 + (T - ramp) * n


# ------------------------------------------------------------------ 64 bits, from the definitions
def exact(case, seed):
    s = _inputs(case, seed, "cuda")
    with torch.no_grad():
        return {"attn": _exact_attn, "step": _exact_step, "append": _exact_append}[case["op"]](case, s)


def _weights(q, k, scale, visible):
    """softmax of scale q k^T over the visible keys by way of its log, in 64 bits; rows without any are zero."""
    z = torch.where(visible, (q @ k.T) * scale, torch.full((), -math.inf, dtype=torch.float64, device=q.device))
    norm = torch.logsumexp(z, -1, keepdim=True)
    return torch.exp(z - torch.where(torch.isinf(norm), torch.zeros_like(norm), norm))


def _exact_attn(c, s):
    B, H, Hk, T, S = c["B"], c["H"], c["Hk"], c["T"], c["S"]
    q, k, v = s["q"].double(), s["k"].double(), s["v"].double()
    d = c["dk"] // 2 if c["diff"] else c["dk"]
    scale = 1 / math.sqrt(d)
    col, row = torch.arange(S, device=q.device)[None, :], torch.arange(T, device=q.device)[:, None]
    train = c["do"] == "train"
    o = torch.zeros(B, H, T, c["dv"], dtype=torch.float64, device=q.device)
    if train:
        do = s["do"].double()
        dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
        dlam = torch.zeros(H, dtype=torch.float64, device=q.device)
    for b in range(B):
        visible = (col < _lens(c)[b]).expand(T, S)
        if c["causal"]:
            visible = visible & (col - row <= S - T)
        for h in range(H):
            n = h * Hk // H
            weight = [1.0, -float(s["lam"][h])] if c["diff"] else [1.0]
            for m, w in enumerate(weight):
                part = slice(m * d, (m + 1) * d)
                A = _weights(q[b, h, :, part], k[b, n, :, part], scale, visible)
                y = A @ v[b, n]
                o[b, h] += w * y
                if train:
                    g = do[b, h] @ v[b, n].T
                    mean = (do[b, h] * y).sum(-1, keepdim=True)
                    if m == 1:
                        dlam[h] -= mean.sum()
                    dz = w * scale * A * (g - mean)
                    dq[b, h, :, part] = dz @ k[b, n, :, part]
                    dk[b, n, :, part] += dz.T @ q[b, h, :, part]
                    dv[b, n] += w * (A.T @ do[b, h])
    out = {"o": o}
    if train:
        out.update(dv=dv, dq=dq, dk=dk)
        if c["diff"]:
            out["dlam"] = dlam
    return out


def _exact_store(c, s, counts):
    """The caches as they are after the call."""
    page, out = c["page"], []
    for name, new in (("k_cache", s["k"]), ("v_cache", s["v"])):
        cache = s[name].clone()
        for b, (first, n) in enumerate(zip(_lens(c), counts)):
            at = torch.arange(first, first + n, device=cache.device)
            rows = new[b][:, None] if new.dim() == 3 else new[b, :, :n]
            cache.transpose(1, 2)[s["table"][b, at // page].long(), at % page] = rows.transpose(0, 1)
        out.append(cache)
    return out


def _exact_step(c, s):
    H, Hk, page = c["H"], c["Hk"], c["page"]
    kc, vc = _exact_store(c, s, [1] * c["B"])
    d = c["dk"] // 2 if c["diff"] else c["dk"]
    o = torch.zeros(c["B"], H, c["dv"], dtype=torch.float64, device=kc.device)
    for b, n in enumerate(_lens(c)):
        at = torch.arange(n + 1, device=kc.device)
        pages, rows = s["table"][b, at // page].long(), at % page
        k, v = kc.transpose(1, 2)[pages, rows].double(), vc.transpose(1, 2)[pages, rows].double()  # [n+1,Hk,..]
        for g in range(Hk):
            heads = slice(g * H // Hk, (g + 1) * H // Hk)
            q = s["q"][b, heads].double()
            visible = torch.ones(1, 1, dtype=torch.bool, device=kc.device)
            y = _weights(q[:, :d], k[:, g, :d], d ** -0.5, visible) @ v[:, g]
            if c["diff"]:
                y = y - s["lam"][heads, None].double() * (_weights(q[:, d:], k[:, g, d:], d ** -0.5, visible) @ v[:, g])
            o[b, heads] = y
    return {"o": o, "k_cache": kc.double(), "v_cache": vc.double()}


def _exact_append(c, s):
    kc, vc = _exact_store(c, s, _counts(c))
    return {"k_cache": kc.double(), "v_cache": vc.double()}

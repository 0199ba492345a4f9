"""GPU parity of whole-sequence attention, ordinary and differential, and its
gradients against the fp64 CPU oracle, element by element within the bounds that
attention_bounds derives."""
import math

import pytest
import torch

import oracle
import retnet_retention_chunkwise_amd as ret
from attention_bounds import bounds, close
from helpers import rel_l2, say, tol

pytestmark = pytest.mark.gpu

DEV = "cuda"
F32, BF16 = torch.float32, torch.bfloat16


def rnd(g, *shape, dtype=F32, scale=1.0, shift=0.0):
    return (torch.randn(shape, generator=g) * scale + shift).to(dtype)


def make(B, H, Hk, T, S, dk, dv, dtype, two, seed=0, sharp=1.5):
    g = torch.Generator().manual_seed(seed + B + H + T + S + dk + dv)
    q, k, v = rnd(g, B, H, T, dk, dtype=dtype, scale=sharp), rnd(g, B, Hk, S, dk, dtype=dtype), rnd(g, B, Hk, S, dv, dtype=dtype)
    return q, k, v, rnd(g, H, scale=0.3, shift=0.6) if two else None, rnd(g, B, H, T, dv, dtype=dtype)


def dev(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


def check(name, q, k, v, lam, do, got, kept=None, grads=None, few=False, **mask):
    """got, kept, grads: what the calls returned, against the oracle's values."""
    lim = bounds(q, k, v, lam, grad_o=do if grads is not None else None, few=few, **mask)
    o, lse, second = oracle.attention(q, k, v, lam, **mask)
    close(name + " o", got, o, lim["o"])
    if kept is not None:
        close(name + " lse", kept[0], lse, lim["lse"])
        if lam is not None:
            close(name + " second", kept[1], second, lim["second"])
    if grads is not None:
        want = oracle.attention_backward(q, k, v, do, lam, **mask)
        for n, g, w in zip(("gq", "gk", "gv", "gl"), grads, want):
            if w is None:
                assert g is None
            else:
                close(f"{name} {n}", g, w, lim[n])


def run(q, k, v, lam, do, **mask):
    a = dev(q, k, v, lam, do)
    m = dict(mask)
    if m.get("lens") is not None:
        m["lens"] = m["lens"].to(DEV)
    o, kept = ret.attention_fwd(*a[:4], keep=True, **m)
    plain = ret.attention_fwd(*a[:4], **m)
    assert torch.equal(o, plain)
    return o, kept, ret.attention_bwd(a[0], a[1], a[2], o, a[4], kept, a[3], **m)


CASES = [
    # B, H, Hk, T, S, dk, dv, dtype, two maps, causal
    (1, 1, 1, 1, 1, 2, 1, F32, True, True),
    (1, 1, 1, 1, 1, 1, 1, BF16, False, False),
    (2, 3, 1, 5, 5, 6, 7, F32, True, True),
    (2, 4, 2, 33, 33, 32, 16, BF16, True, True),
    (1, 2, 2, 64, 64, 64, 64, BF16, True, False),
    (1, 2, 1, 65, 97, 34, 33, F32, True, True),
    (2, 2, 2, 130, 130, 64, 64, F32, False, True),
    (1, 3, 3, 129, 129, 41, 63, BF16, False, True),
    (1, 4, 1, 200, 200, 128, 128, BF16, True, True),
    (2, 2, 1, 77, 301, 128, 100, BF16, False, False),
    (1, 2, 2, 150, 150, 130, 129, F32, True, True),
    (1, 2, 1, 257, 257, 256, 256, BF16, True, True),
    (1, 2, 2, 100, 100, 256, 40, BF16, False, True),
    (1, 2, 1, 70, 90, 256, 256, F32, True, False),
    (1, 1, 1, 40, 40, 255, 255, F32, False, True),
    (3, 8, 8, 16, 16, 48, 24, BF16, True, True),
    (1, 2, 1, 190, 190, 192, 96, BF16, True, True),   # one side wider than the other
    (1, 2, 2, 175, 175, 64, 160, BF16, True, False),
    (1, 2, 2, 140, 140, 192, 128, BF16, False, True),
    (1, 2, 1, 70, 70, 160, 64, F32, True, True),
    (1, 2, 1, 70, 70, 96, 256, F32, False, True),
    (1, 2, 2, 300, 20, 64, 64, BF16, True, True),   # more rows than keys: the first see none
    (1, 2, 1, 20, 300, 64, 64, BF16, True, True),   # the last rows of a longer sequence
]


@pytest.mark.parametrize("B,H,Hk,T,S,dk,dv,dtype,two,causal", CASES)
def test_matches_oracle(B, H, Hk, T, S, dk, dv, dtype, two, causal):
    name = f"attention B{B} H{H}/{Hk} T{T} S{S} dk{dk} dv{dv} {dtype} maps={1 + two} causal={causal}"
    say(name)
    q, k, v, lam, do = make(B, H, Hk, T, S, dk, dv, dtype, two)
    o, kept, grads = run(q, k, v, lam, do, causal=causal)
    check(name, q, k, v, lam, do, o, kept, grads, causal=causal)
    again = run(q, k, v, lam, do, causal=causal)
    assert torch.equal(o, again[0]) and all(x is y or torch.equal(x, y) for x, y in zip(grads, again[2]))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("two", [True, False])
@pytest.mark.parametrize("B,H,Hk,T,S,dk,dv", [(1, 2, 1, 1, 700, 64, 64), (2, 4, 2, 16, 2049, 32, 40), (1, 1, 1, 3, 1024, 128, 128),
                                              (1, 2, 2, 70, 1500, 128, 256), (2, 2, 1, 300, 530, 100, 72)])
def test_few_rows_over_many_keys(B, H, Hk, T, S, dk, dv, two, dtype):
    """The keys are split over workgroups and joined."""
    name = f"split B{B} H{H}/{Hk} T{T} S{S} dk{dk} dv{dv} {dtype} maps={1 + two}"
    say(name)
    q, k, v, lam, do = make(B, H, Hk, T, S, dk, dv, dtype, two)
    assert ret.load().retention_attention_workspace_bytes(B, H, Hk, T, S, dk, dv, 1 + two, int(dtype == BF16)) > 0
    for mask in (dict(causal=True), dict(causal=False, lens=torch.tensor([S // 3] + [0] * (B - 1), dtype=torch.int32))):
        o, kept, grads = run(q, k, v, lam, do, **mask)
        check(name, q, k, v, lam, do, o, kept, grads, **mask)


@pytest.mark.parametrize("two", [True, False])
@pytest.mark.parametrize("T,S,d,dv,lens", [(1, 1, 64, 64, None), (2, 2, 64, 64, None), (3, 3, 96, 128, [3, 2]), (9, 9, 100, 36, None),
                                           (32, 32, 128, 128, [32, 0]), (70, 31, 256, 256, None), (40, 100, 64, 64, [32, 7])])
def test_gradients_over_few_keys(T, S, d, dv, lens, two):
    """bf16 rows that see at most 32 keys: what dP - D leaves is not lost to the rounding of o."""
    for causal in (True, False):
        name = f"few T{T} S{S} dk{d} dv{dv} lens={lens} maps={1 + two} causal={causal}"
        say(name)
        q, k, v, lam, do = make(2, 4, 2, T, S, d, dv, BF16, two)
        mask = dict(causal=causal, lens=None if lens is None else torch.tensor(lens, dtype=torch.int32))
        o, kept, grads = run(q, k, v, lam, do, **mask)
        check(name, q, k, v, lam, do, o, kept, grads, few=True, **mask)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("B,H,Hk,T,S,dk,dv,causal", [(1, 2, 1, 600, 40, 256, 256, False), (1, 3, 1, 520, 130, 60, 72, True)])
def test_rows_shared_out(B, H, Hk, T, S, dk, dv, causal, dtype):
    """Few keys that many rows see: the rows are shared out over workgroups and their sums added."""
    say(f"shared out T{T} S{S} dk{dk} dv{dv} {dtype}")
    for two in (True, False):
        q, k, v, lam, do = make(B, H, Hk, T, S, dk, dv, dtype, two)
        o, kept, grads = run(q, k, v, lam, do, causal=causal, offset=0)
        check(f"shared out maps={1 + two}", q, k, v, lam, do, o, kept, grads, causal=causal, offset=0)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("causal,offset", [(False, None), (True, 0), (True, 9), (True, -40), (True, -500), (True, 500)])
def test_masks(dtype, causal, offset):
    """Lengths beyond, at and below zero, offsets that leave rows without keys; what is masked holds NaN and infinities."""
    B, H, Hk, T, S, dk, dv = 5, 4, 2, 100, 110, 64, 48
    lens = torch.tensor([110, 64, 1, 0, 33], dtype=torch.int32)
    say(f"masks {dtype} causal={causal} offset={offset}")
    q, k, v, lam, do = make(B, H, Hk, T, S, dk, dv, dtype, True)
    for b, n in enumerate(lens.tolist()):
        k[b, :, n:] = float("nan")
        v[b, :, n:] = float("inf") if b % 2 else float("nan")
    mask = dict(causal=causal, offset=offset, lens=lens)
    o, kept, grads = run(q, k, v, lam, do, **mask)
    check("masks", q, k, v, lam, do, o, kept, grads, **mask)
    for b, n in enumerate(lens.tolist()):
        assert (grads[1][b, :, n:] == 0).all() and (grads[2][b, :, n:] == 0).all()
    # lengths out of range are taken into it
    far = torch.tensor([1000, 64, 1, -7, 33], dtype=torch.int32)
    p, _, more = run(q, k, v, lam, do, causal=causal, offset=offset, lens=far)
    assert torch.equal(o, p) and all(torch.equal(x, y) for x, y in zip(grads, more))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_no_tokens(dtype):
    q, k, v, lam, do = dev(*make(2, 4, 2, 0, 9, 16, 8, dtype, True))
    o, kept = ret.attention_fwd(q, k, v, lam, keep=True)
    gq, gk, gv, gl = ret.attention_bwd(q, k, v, o, do, kept, lam)
    assert o.shape == (2, 4, 0, 8) and gq.shape == q.shape
    assert all((g == 0).all() for g in (gk, gv, gl))
    q, k, v, lam, do = dev(*make(2, 4, 2, 9, 0, 16, 8, dtype, True))
    o, kept = ret.attention_fwd(q, k, v, lam, keep=True, causal=False)
    gq, gk, gv, gl = ret.attention_bwd(q, k, v, o, do, kept, lam, causal=False)
    assert (o == 0).all() and (gq == 0).all() and (gl == 0).all() and torch.isneginf(kept[0]).all() and gk.numel() == 0


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_sharp_and_flat_rows(dtype):
    """Scores of hundreds, growing along the keys (the running maximum moves every tile) and equal ones."""
    q, k, v, lam, do = make(1, 2, 1, 90, 200, 64, 32, dtype, True, sharp=1.0)
    k = (k.float() * torch.linspace(0.1, 6, 200)[:, None]).to(dtype)
    q = (q.float() * 8).to(dtype)
    q[:, 1] = 0  # every key alike
    o, kept, grads = run(q, k, v, lam, do, causal=False)
    check("sharp", q, k, v, lam, do, o, kept, grads, causal=False)
    # one key takes all: the output is its value exactly
    q, k = torch.zeros(1, 1, 3, 8, dtype=dtype), torch.zeros(1, 1, 150, 8, dtype=dtype)
    q[..., 0], k[:, :, 77, 0] = 60, 60
    v = make(1, 1, 1, 3, 150, 8, 5, dtype, False)[2]
    got = ret.attention_fwd(*dev(q, k, v), causal=False)
    assert torch.equal(got.cpu(), v[:, :, 77:78].expand(1, 1, 3, 5))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_scale_and_not_finite(dtype):
    q, k, v, lam, do = make(1, 2, 2, 50, 50, 32, 16, dtype, True)
    o, kept, grads = run(q, k, v, lam, do, scale=0.02)
    check("scale", q, k, v, lam, do, o, kept, grads, scale=0.02)
    q[0, 1, 7, 3] = float("nan")
    got = ret.attention_fwd(*dev(q, k, v, lam)).cpu()
    assert torch.isnan(got[0, 1, 7]).all()
    got[0, 1, 7] = o.cpu()[0, 1, 7]
    assert torch.isfinite(got).all()


def strided(t, how):
    """A copy of t [B,H,T,d] on the device in another layout."""
    t = t.to(DEV)
    if how == "token":  # [B,T,H,d]
        return t.transpose(1, 2).contiguous().transpose(1, 2)
    if how == "slice":  # the middle of wider rows, at an odd element
        wide = torch.full((*t.shape[:-1], t.shape[-1] + 5), float("nan"), dtype=t.dtype, device=DEV)
        wide[..., 3:3 + t.shape[-1]] = t
        return wide[..., 3:3 + t.shape[-1]]
    return t


@pytest.mark.parametrize("how", ["token", "slice"])
@pytest.mark.parametrize("dtype,dk,dv", [(F32, 20, 12), (BF16, 64, 64), (BF16, 30, 129)])
def test_layouts(how, dtype, dk, dv):
    """Other strides and alignments give the same bits, and what lies between rows stays."""
    say(f"layout {how} {dtype} dk{dk} dv{dv}")
    ts = make(2, 4, 2, 70, 70, dk, dv, dtype, True)
    o, kept, grads = run(*ts)
    q, k, v, do = (strided(t, how) for t in (ts[0], ts[1], ts[2], ts[4]))
    lam = ts[3].to(DEV)
    out = strided(torch.zeros_like(ts[4]), how)
    outs = [strided(torch.zeros_like(t), how) for t in ts[:3]]
    p, kept2 = ret.attention_fwd(q, k, v, lam, keep=True, o=out)
    more = ret.attention_bwd(q, k, v, p, do, kept2, lam, grad_q=outs[0], grad_k=outs[1], grad_v=outs[2])
    assert p is out and all(x is y for x, y in zip(outs, more[:3]))
    for x, y in zip((o, *kept, *grads), (p, *kept2, *more)):
        assert torch.equal(x, y)
    if how == "slice":
        for t in (out, *outs):
            whole = t.as_strided((*t.shape[:-1], t.shape[-1] + 5), t.stride(), t.storage_offset() - 3)
            assert torch.isnan(whole[..., :3]).all() and torch.isnan(whole[..., 3 + t.shape[-1]:]).all()


def test_slices_of_one_projection():
    """q, k and v as columns of one fused projection [B,T,(H + 2 Hk) d], gradients into one like it."""
    B, H, Hk, T, d = 2, 4, 2, 60, 32
    g = torch.Generator().manual_seed(3)
    fused = rnd(g, B, T, (H + 2 * Hk) * d, dtype=BF16).to(DEV)

    def parts(t):
        heads = t.view(B, T, H + 2 * Hk, d).transpose(1, 2)
        return heads[:, :H], heads[:, H:H + Hk], heads[:, H + Hk:]

    q, k, v = parts(fused)
    do = rnd(g, B, H, T, d, dtype=BF16).to(DEV)
    grad = torch.full_like(fused, float("nan"))
    o, kept = ret.attention_fwd(q, k, v, keep=True)
    gq, gk, gv = parts(grad)
    ret.attention_bwd(q, k, v, o, do, kept, grad_q=gq, grad_k=gk, grad_v=gv)
    check("fused", q.cpu(), k.cpu(), v.cpu(), None, do.cpu(), o, kept, (gq, gk, gv, None))


def test_shared_heads_sum_their_gradients():
    """Gradients of shared keys are those of copies for every head, added."""
    q, k, v, lam, do = dev(*make(2, 6, 2, 90, 90, 32, 32, F32, True))
    o, kept = ret.attention_fwd(q, k, v, lam, keep=True)
    _, gk, gv, gl = ret.attention_bwd(q, k, v, o, do, kept, lam)
    kk, vv = k.repeat_interleave(3, 1), v.repeat_interleave(3, 1)
    o2, kept2 = ret.attention_fwd(q, kk, vv, lam, keep=True)
    assert torch.equal(o, o2)
    _, gk2, gv2, gl2 = ret.attention_bwd(q, kk, vv, o2, do, kept2, lam)
    assert torch.equal(gl, gl2)
    for a, b in ((gk, gk2), (gv, gv2)):
        assert rel_l2(a, b.view(2, 2, 3, 90, 32).sum(2)) < 1e-6


def test_gradients_by_differences():
    """The loss along random directions, in fp32: central differences of the call itself."""
    q, k, v, lam, do = dev(*make(1, 2, 1, 40, 40, 16, 16, F32, True))
    o, kept = ret.attention_fwd(q, k, v, lam, keep=True)
    grads = ret.attention_bwd(q, k, v, o, do, kept, lam)
    g = torch.Generator().manual_seed(11)
    loss = lambda a: float((do.double() * ret.attention_fwd(*a).double()).sum())  # noqa: E731
    h = 2.0 ** -6
    for i, t in enumerate((q, k, v, lam)):
        step = torch.randn(t.shape, generator=g).to(DEV)
        at = [q, k, v, lam]
        at[i] = t + h * step
        a = loss(at)
        at[i] = t - h * step
        b = loss(at)
        want = float((grads[i].double() * step.double()).sum())
        # the difference's own error: h^2 / 6 of the third derivative (below 60 for these sizes), and
        # 2^-24 of the outputs' magnitudes, sum |do| |o|, over h
        size = float((do.abs() * o.abs()).sum())
        assert abs((a - b) / (2 * h) - want) < 60 * h * h / 6 * max(1.0, abs(want)) + 2.0 ** -22 * size / h


@pytest.mark.parametrize("B,H,Hk,T,S,dk,dv,dtype,two,causal", [
    (2, 8, 2, 2048, 2048, 128, 128, BF16, True, True), (1, 4, 4, 1500, 1500, 256, 256, BF16, True, True),
    (1, 4, 2, 1111, 1111, 64, 64, BF16, False, False), (1, 4, 2, 1111, 1111, 128, 128, F32, True, True)])
def test_long_sequences(B, H, Hk, T, S, dk, dv, dtype, two, causal):
    say(f"long B{B} H{H}/{Hk} T{T} dk{dk} dv{dv} {dtype}")
    ts = make(B, H, Hk, T, S, dk, dv, dtype, two)
    o, kept, grads = run(*ts, causal=causal)
    want = oracle.attention(*ts[:4], causal=causal)
    assert rel_l2(o, want[0]) <= tol(dtype) and rel_l2(kept[0], want[1]) <= 1e-6
    for g, w in zip(grads, oracle.attention_backward(*ts[:3], ts[4], ts[3], causal=causal)):
        assert w is None or rel_l2(g, w) <= tol(dtype)
    if two:
        assert rel_l2(grads[3], oracle.attention_backward(*ts[:3], ts[4], ts[3], causal=causal)[3]) <= 1e-5


@pytest.mark.parametrize("T,S", [(150, 150), (16, 1500)])
def test_graph_and_streams(T, S):
    """Captured and replayed, in two graphs with workspaces of their own, and on another stream: the eager bits."""
    ts = make(2, 4, 2, T, S, 64, 64, BF16, True)
    q, k, v, lam, do = dev(*ts)
    o, kept = ret.attention_fwd(q, k, v, lam, keep=True)
    want = (o, *kept, *ret.attention_bwd(q, k, v, o, do, kept, lam))

    def both():
        o, kept = ret.attention_fwd(q, k, v, lam, keep=True)
        return (o, *kept, *ret.attention_bwd(q, k, v, o, do, kept, lam))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = both()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            graphs.append((graph, both()))
    for _ in range(3):
        for _, held in graphs:
            for t in held:
                t.fill_(float("nan"))
        for graph, _ in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for _, held in graphs:
            assert all(torch.equal(a, b) for a, b in zip(held, want))
        both()
        torch.cuda.synchronize()


def test_two_streams_at_once():
    """Training passes of different inputs that overlap in time, each with workspaces of its own: the bits of each alone."""
    sets = [dev(*make(1, 4, 2, 700, 700, d, 64, dtype, True, seed=d)) for d, dtype in ((64, BF16), (96, F32))]

    def both(q, k, v, lam, do):
        o, kept = ret.attention_fwd(q, k, v, lam, keep=True)
        return (o, *kept, *ret.attention_bwd(q, k, v, o, do, kept, lam))

    want = [both(*s) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(both(*sets[i]))
    torch.cuda.synchronize()
    for i, w in enumerate(want):
        assert all(torch.equal(a, b) for run in got[i] for a, b in zip(run, w))


@pytest.mark.parametrize("seed", range(16))
def test_random_shapes(seed):
    """Any widths, lengths, masks and types, against the bounds."""
    g = torch.Generator().manual_seed(seed)
    pick = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=g))  # noqa: E731
    two, dtype = bool(seed & 1), BF16 if seed & 2 else F32
    Hk, B = pick(1, 3), pick(1, 2)
    H, T, S = Hk * pick(1, 4), pick(1, 200), pick(1, 600)
    dk, dv = (2 * pick(1, 128) if two else pick(1, 256)), pick(1, 256)
    if seed & 4:
        dk, dv = -(-dk // 16) * 16, -(-dv // 8) * 8
    mask = dict(causal=bool(seed & 8))
    if mask["causal"]:
        mask["offset"] = pick(-T, S)
    if pick(0, 1):
        mask["lens"] = torch.tensor([pick(0, S) for _ in range(B)], dtype=torch.int32)
    name = f"random {seed}: B{B} H{H}/{Hk} T{T} S{S} dk{dk} dv{dv} {dtype} maps={1 + two} {mask}"
    say(name)
    q, k, v, lam, do = make(B, H, Hk, T, S, dk, dv, dtype, two, seed=seed)
    o, kept, grads = run(q, k, v, lam, do, **mask)
    check(name, q, k, v, lam, do, o, kept, grads, **mask)

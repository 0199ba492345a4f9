"""GPU parity of the decode step over a paged cache and of the cache's filling
against the fp64 CPU oracle, and of prompts, fillings and steps together."""
import pytest
import torch

import oracle
import retnet_retention_chunkwise_amd as ret
from attention_bounds import bounds, close
from helpers import say

pytestmark = pytest.mark.gpu

DEV = "cuda"
F32, BF16, I32 = torch.float32, torch.bfloat16, torch.int32


def rnd(g, *shape, dtype=F32, scale=1.0, shift=0.0):
    return (torch.randn(shape, generator=g) * scale + shift).to(dtype)


def make(lens, H, Hk, dk, dv, page, dtype, two, spare=2, most=None, seed=0):
    """Inputs of a step over sequences of the given lengths, pages in random order, NaN where no token is."""
    B = len(lens)
    most = -(-(max(lens) + 1) // page) if most is None else most
    g = torch.Generator().manual_seed(seed + B + H + dk + dv + page)
    P = B * most + spare
    kc, vc = rnd(g, P, Hk, page, dk, dtype=dtype), rnd(g, P, Hk, page, dv, dtype=dtype)
    table = torch.randperm(P, generator=g)[:B * most].view(B, most).to(I32)
    used = torch.zeros(P, page, dtype=torch.bool)
    for b, n in enumerate(lens):
        for s in range(max(n, 0)):
            if s < most * page:
                used[table[b, s // page], s % page] = True
    kc.transpose(1, 2)[~used] = float("nan")
    vc.transpose(1, 2)[~used] = float("inf")
    q, k, v = rnd(g, B, H, dk, dtype=dtype, scale=1.5), rnd(g, B, Hk, dk, dtype=dtype), rnd(g, B, Hk, dv, dtype=dtype)
    lam = rnd(g, H, scale=0.3, shift=0.6) if two else None
    return q, k, v, kc, vc, table, torch.tensor(lens, dtype=I32), lam


def same(a, b):
    return torch.equal(torch.nan_to_num(a.cpu().float(), 7, 8, 9), torch.nan_to_num(b.cpu().float(), 7, 8, 9))


def check(name, q, k, v, kc, vc, table, lens, lam, got, got_kc, got_vc):
    o, want_kc, want_vc = oracle.attention_step(q, k, v, kc, vc, table, lens, lam)
    lim = torch.zeros_like(o)
    pages, page, most = kc.shape[0], kc.shape[2], table.shape[1]
    for b in range(q.shape[0]):
        n = int(lens[b])
        if n < 0:
            continue
        at = [(int(table[b, s // page]), s % page) for s in range(min(n, most * page)) if 0 <= int(table[b, s // page]) < pages]
        ks = torch.stack([kc[p, :, r] for p, r in at] + [k[b]], 1)[None]
        vs = torch.stack([vc[p, :, r] for p, r in at] + [v[b]], 1)[None]
        lim[b] = bounds(q[b:b + 1, :, None], ks, vs, lam, causal=False)["o"][0, :, 0]
    close(name, got, o, lim)
    assert same(got_kc, want_kc) and same(got_vc, want_vc), name


def run(name, q, k, v, kc, vc, table, lens, lam):
    dq, dk, dv, dkc, dvc, dt, dl, dlam = (None if t is None else t.to(DEV) for t in (q, k, v, kc, vc, table, lens, lam))
    got = ret.attention_step(dq, dk, dv, dkc, dvc, dt, dl, dlam)
    check(name, q, k, v, kc, vc, table, lens, lam, got, dkc, dvc)
    again = ret.attention_step(dq, dk, dv, dkc, dvc, dt, dl, dlam)  # the same call again: nothing has moved
    assert torch.equal(got, again)
    return got


@pytest.mark.parametrize("two", [True, False])
@pytest.mark.parametrize("lens,H,Hk,dk,dv,page,dtype", [
    ([0], 1, 1, 2, 1, 1, F32),
    ([0, 1, 31, 32, 33], 2, 1, 6, 7, 5, F32),
    ([5, 0, 100], 4, 2, 32, 16, 16, BF16),
    ([64, 127, 3], 6, 3, 64, 64, 64, BF16),
    ([200, 17], 8, 1, 34, 33, 24, F32),
    ([90, 600], 16, 1, 128, 128, 16, BF16),
    ([40, 129], 20, 1, 64, 40, 32, BF16),       # more query heads than one workgroup takes
    ([300, 0, 77], 4, 4, 256, 256, 100, BF16),
    ([150, 31], 2, 2, 256, 256, 7, F32),
    ([1, 700], 34, 2, 18, 130, 1, BF16),
    ([2000, 1023, 1024], 4, 2, 128, 100, 64, F32),
    ([511, 1200], 3, 3, 40, 256, 256, BF16),
    ([33, 700], 4, 1, 192, 96, 64, BF16),
    ([20, 333], 2, 2, 160, 68, 16, F32),
    ([65, 130], 4, 2, 64, 136, 64, F32),
])
def test_step_matches_oracle(lens, H, Hk, dk, dv, page, dtype, two):
    name = f"step {lens} H{H}/{Hk} dk{dk} dv{dv} page{page} {dtype} maps={1 + two}"
    say(name)
    run(name, *make(lens, H, Hk, dk, dv, page, dtype, two))


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_step_masks(dtype):
    """Idle sequences, full caches, pages that are not there (also the new token's), a table wider than needed."""
    lens = [70, -1, 96, 33, 1000, 60, -5]
    args = make(lens, 4, 2, 32, 24, 16, dtype, True, most=6)
    q, k, v, kc, vc, table, n, lam = args
    table[0, 2], table[5, 0], table[5, 1], table[3, 2] = -1, 1 << 30, kc.shape[0], -7
    say(f"step masks {dtype}")
    got = run("step masks", *args)
    assert (got[1] == 0).all() and (got[6] == 0).all()
    for most, split in ((6, False), (600, True)):  # the same with the keys split over workgroups
        wide = torch.full((len(lens), most), -1, dtype=I32)
        wide[:, :6] = table
        assert (ret.load().retention_attention_step_workspace_bytes(7, 4, 2, 32, 24, 16, most, 2, int(dtype == BF16)) > 0) == split
        m = n.clone()
        m[2], m[4] = 95, 95
        run(f"step masks, {most} pages", q, k, v, kc, vc, wide, m, lam)
    run("no pages at all", q, k, v, kc, vc, torch.empty(7, 0, dtype=I32), n, lam)
    run("no page is there", q, k, v, kc[:0], vc[:0], table, n, lam)


def test_step_layouts():
    """Token-major pages, and rows inside wider ones at odd elements: the same bits, nothing else touched."""
    for dtype, dk, dv in ((BF16, 32, 48), (BF16, 30, 17), (F32, 20, 12)):
        say(f"step layouts {dtype} dk{dk} dv{dv}")
        args = [None if t is None else t.to(DEV) for t in make([100, 3, 40], 4, 2, dk, dv, 16, dtype, True)]
        q, k, v, kc, vc, table, lens, lam = args
        token = [t.transpose(1, 2).contiguous().transpose(1, 2) for t in (kc, vc)]

        def wide(t):
            w = torch.full((*t.shape[:-1], t.shape[-1] + 5), 3.0, dtype=t.dtype, device=DEV)
            w[..., 3:-2] = t
            return w, w[..., 3:-2]

        wides = [wide(t) for t in (kc, vc, q, k, v)]
        o = ret.attention_step(q, k, v, kc, vc, table, lens, lam)
        a = ret.attention_step(q, k, v, *token, table, lens, lam)
        out = wide(torch.zeros_like(o))
        b = ret.attention_step(wides[2][1], wides[3][1], wides[4][1], wides[0][1], wides[1][1], table, lens, lam, o=out[1])
        assert b is out[1] and torch.equal(o, a) and torch.equal(o, b)
        for i, t in enumerate((kc, vc)):
            assert same(t, token[i]) and same(t, wides[i][1])
        for w, _ in (*wides, out):
            assert (w[..., :3] == 3).all() and (w[..., -2:] == 3).all()


def test_step_in_a_cache_beyond_32_bits():
    """Pages whose elements lie past 2^31 and 2^32 bytes."""
    P, Hk, page, d = 70000, 2, 256, 64  # 2.3e9 elements, 4.6 GB each
    g = torch.Generator().manual_seed(1)
    kc, vc = (torch.empty(P, Hk, page, d, dtype=BF16, device=DEV) for _ in range(2))
    table = torch.tensor([[P - 1, 3, P - 2], [65535, 65536, 40000]], dtype=I32)
    lens = torch.tensor([700, 600], dtype=I32)
    keys, vals = rnd(g, 2, Hk, 700, d, dtype=BF16), rnd(g, 2, Hk, 700, d, dtype=BF16)
    q, k, v = rnd(g, 2, 4, d, dtype=BF16), rnd(g, 2, Hk, d, dtype=BF16), rnd(g, 2, Hk, d, dtype=BF16)
    say("step beyond 32 bits")
    ret.cache_append(keys.to(DEV), vals.to(DEV), kc, vc, table.to(DEV), torch.zeros(2, dtype=I32, device=DEV), lens.to(DEV))
    got = ret.attention_step(q.to(DEV), k.to(DEV), v.to(DEV), kc, vc, table.to(DEV), lens.to(DEV))
    used = table.flatten().tolist()
    small = {p: i for i, p in enumerate(used)}
    at = torch.tensor(used, device=DEV)
    skc, svc = kc[at].cpu(), vc[at].cpu()
    t2 = torch.tensor([[small[int(p)] for p in row] for row in table], dtype=I32)
    for b in range(2):
        n = int(lens[b])
        ks = torch.cat([keys[b, :, :n], k[b][:, None]], 1)[None]
        vs = torch.cat([vals[b, :, :n], v[b][:, None]], 1)[None]
        want = oracle.attention(q[b:b + 1, :, None], ks, vs, causal=False)[0][0, :, 0]
        close(f"sequence {b}", got[b], want, bounds(q[b:b + 1, :, None], ks, vs, causal=False)["o"][0, :, 0])
        p, r = t2[b, n // page], n % page
        assert torch.equal(skc[p, :, r], k[b]) and torch.equal(svc[p, :, r], v[b])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("Hk,T,dk,dv,page", [(1, 1, 1, 1, 1), (2, 9, 3, 5, 4), (2, 70, 32, 40, 16), (3, 33, 129, 200, 7),
                                             (2, 130, 256, 64, 100)])
def test_append_matches_oracle(Hk, T, dk, dv, page, dtype):
    B, most = 5, -(-(T + 20) // page)
    say(f"append Hk{Hk} T{T} dk{dk} dv{dv} page{page} {dtype}")
    g = torch.Generator().manual_seed(T + dk)
    P = B * most + 1
    kc, vc = rnd(g, P, Hk, page, dk, dtype=dtype), rnd(g, P, Hk, page, dv, dtype=dtype)
    k, v = rnd(g, B, Hk, T, dk, dtype=dtype), rnd(g, B, Hk, T, dv, dtype=dtype)
    table = torch.randperm(P, generator=g)[:B * most].view(B, most).to(I32)
    table[4, most // 2] = -1
    start = torch.tensor([0, 7, -1, most * page - 2, 3], dtype=I32)  # one idle, one that runs out of pages
    for counts in (None, torch.tensor([T, max(T - 3, 0), T, T + 9, -2], dtype=I32)):
        want = oracle.cache_append(k, v, kc, vc, table, start, counts)
        a, b = kc.to(DEV), vc.to(DEV)
        ret.cache_append(k.to(DEV), v.to(DEV), a, b, table.to(DEV), start.to(DEV), None if counts is None else counts.to(DEV))
        assert torch.equal(a.cpu(), want[0]) and torch.equal(b.cpu(), want[1])
        # token-major prompts and pages, slices of wider rows
        tok = lambda t: t.to(DEV).transpose(1, 2).contiguous().transpose(1, 2)  # noqa: E731
        a, b = tok(kc), tok(vc)
        both = torch.cat([tok(k).transpose(1, 2), tok(v).transpose(1, 2)], -1).transpose(1, 2)
        ret.cache_append(both[..., :dk], both[..., dk:], a, b, table.to(DEV), start.to(DEV),
                         None if counts is None else counts.to(DEV))
        assert torch.equal(a.cpu(), want[0]) and torch.equal(b.cpu(), want[1])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("two", [True, False])
def test_prompt_then_steps(two, dtype):
    """A padded batch of prompts, its keys into the cache, then steps: every row as one causal call gives it."""
    B, H, Hk, dk, dv, page, steps = 3, 4, 2, 64, 48, 16, 20
    lens = [100, 37, 1]
    n = max(lens) + steps
    say(f"prompt then steps maps={1 + two} {dtype}")
    g = torch.Generator().manual_seed(2)
    q, k, v = rnd(g, B, H, n, dk, dtype=dtype), rnd(g, B, Hk, n, dk, dtype=dtype), rnd(g, B, Hk, n, dv, dtype=dtype)
    lam = rnd(g, H, scale=0.3, shift=0.6) if two else None
    dq, dk_, dv_ = q.to(DEV), k.to(DEV), v.to(DEV)
    dlam = None if lam is None else lam.to(DEV)
    want = [oracle.attention(q[b:b + 1], k[b:b + 1], v[b:b + 1], lam)[0][0] for b in range(B)]
    lim = [bounds(q[b:b + 1], k[b:b + 1], v[b:b + 1], lam)["o"][0] for b in range(B)]
    T = max(lens)
    at = torch.tensor(lens, dtype=I32, device=DEV)
    o = ret.attention_fwd(dq[:, :, :T], dk_[:, :, :T], dv_[:, :, :T], dlam, lens=at)
    P = B * -(-n // page)
    table = torch.randperm(P, generator=g).view(B, -1).to(I32).to(DEV)
    kc, vc = torch.full((P, Hk, page, dk), float("nan"), dtype=dtype, device=DEV), torch.full((P, Hk, page, dv), float("nan"),
                                                                                            dtype=dtype, device=DEV)
    ret.cache_append(dk_[:, :, :T], dv_[:, :, :T], kc, vc, table, torch.zeros_like(at), at)
    for b in range(B):
        close(f"prompt {b}", o[b, :, :lens[b]], want[b][:, :lens[b]], lim[b][:, :lens[b]])
    b = torch.arange(B, device=DEV)
    for _ in range(steps):
        i = at.long()
        y = ret.attention_step(dq[b, :, i], dk_[b, :, i], dv_[b, :, i], kc, vc, table, at, dlam)
        for j in range(B):
            close(f"step {int(i[j])}", y[j], want[j][:, int(i[j])], lim[j][:, int(i[j])])
        at += 1


def test_shared_prefix():
    """Sequences that share the pages of a prefix, each storing into a page of its own."""
    q, k, v, kc, vc, table, lens, lam = make([32, 40, 47], 4, 2, 32, 32, 16, BF16, True)
    table[1, :2], table[2, :2] = table[0, :2], table[0, :2]
    run("shared prefix", q, k, v, kc, vc, table, lens, lam)


@pytest.mark.parametrize("most", [4, 300])
def test_step_graph_and_streams(most):
    """One captured decode loop over lengths that move on the device, replayed; and another stream."""
    lens = [10, 0, 37]
    q, k, v, kc, vc, table, n, lam = (t.to(DEV) for t in make(lens, 4, 2, 32, 32, 16, BF16, True, most=4))
    wide = torch.full((3, most), -1, dtype=I32, device=DEV)
    wide[:, :4] = table
    want, at = [], n.clone()
    ka, va = kc.clone(), vc.clone()
    for _ in range(6):
        want.append(ret.attention_step(q, k, v, ka, va, wide, at, lam))
        at += 1
    kb, vb, at = kc.clone(), vc.clone(), n.clone()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = ret.attention_step(q, k, v, kb, vb, wide, at, lam)
        at += 1
    for i in range(6):
        o.fill_(float("nan"))
        graph.replay()
        assert torch.equal(o, want[i])
        ret.attention_step(q, k, v, kc.clone(), vc.clone(), wide, n, lam)
        torch.cuda.synchronize()
    assert same(ka, kb) and same(va, vb)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = ret.attention_step(q, k, v, kc, vc, wide, n, lam)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want[0])


def test_hybrid_block():
    """Retention and differential attention in one block, as a hybrid stack has them: residual norm, mixer, gated
    per-head norm, twice, against the oracle's operators in turn."""
    B, H, T, d = 2, 4, 70, 64
    g = torch.Generator().manual_seed(5)
    x = rnd(g, B, T, H * d)
    z = rnd(g, B, T, H, d)
    w = rnd(g, H, d, scale=0.2, shift=1.0)
    lam = rnd(g, H, scale=0.3, shift=0.6)
    gamma = [0.97, 0.9, 0.8, 0.5]
    heads = lambda t: t.view(B, T, H, d).transpose(1, 2)  # noqa: E731
    xd, zd, wd = x.to(DEV), z.to(DEV), w.to(DEV)
    h = heads(xd).contiguous()
    y, _ = ret.chunkwise_fwd(h / 8, h / 8, h, gamma, 32)
    r, n = ret.residual_norm(xd, ret.group_norm_gated(y, zd, wd).flatten(-2))
    a = ret.attention_fwd(heads(n), heads(n), heads(n), lam.to(DEV))
    out, _ = ret.residual_norm(r, ret.group_norm_gated(a, zd, wd).flatten(-2))

    def up(t):
        return t.double()

    ho = heads(up(x))
    yo, _ = oracle.recurrent(ho / 8, ho / 8, ho, torch.tensor(gamma))
    ro = oracle.residual(x, oracle.group_norm_gated(yo, z, w).flatten(-2))
    no = heads(oracle.stream_norm(ro))
    ao = oracle.attention(no, no, no, lam)[0]
    want = oracle.residual(ro, oracle.group_norm_gated(ao, z, w).flatten(-2))
    err = float((out.cpu().double() - want).norm() / want.norm())
    say(f"hybrid block: rel-L2 {err:.2e}")
    assert err <= 1e-4

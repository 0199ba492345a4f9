"""Every visible key counts once, and with its own value: a key lost, repeated or taken from elsewhere at the border
of a tile, page or share shows in full, where an error bound over hundreds of keys would cover it."""
import pytest
import torch

import oracle
import retnet_retention_chunkwise_amd as ret
from helpers import rel_l2, say

pytestmark = pytest.mark.gpu

DEV = "cuda"
F32, BF16, I32 = torch.float32, torch.bfloat16, torch.int32
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8}
WIDTHS = [(64, 64), (128, 128), (192, 96), (40, 256), (256, 256), (130, 77)]
LAM = 0.375  # its share of a weight and 1 - LAM differ, and both are exact


def pages_of(lens, page, g, spare=2):
    """A table of pages in random order, their number."""
    most = -(-(max(lens) + 1) // page)
    P = len(lens) * most + spare
    return torch.randperm(P, generator=g)[:len(lens) * most].view(len(lens), most).to(I32), P


def share(got, n, maps, dtype, where):
    """got is 1 / n (two maps: (1 - LAM) / n) where a key's channel is, else 0."""
    want = torch.where(where, (1.0 if maps == 1 else 1 - LAM) / n, torch.zeros((), dtype=torch.float64))
    # equal scores: weights are 1, their sums exact; a division, a product and an fp32 sum, then the output's rounding
    assert ((got.cpu().double() - want).abs() <= want * (HALF[dtype] * 1.01 + 8 * 2.0 ** -24)).all()


@pytest.mark.parametrize("two", [True, False])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dk,dv", WIDTHS)
@pytest.mark.parametrize("T,S,causal", [(3, 1100, False), (70, 513, True), (129, 129, True), (1, 1, False)])
def test_forward_counts_each_key(T, S, causal, dk, dv, dtype, two):
    """q = 0 weighs the visible keys alike; one key at a time has a channel of its own."""
    say(f"each key T{T} S{S} dk{dk} dv{dv} {dtype} maps={1 + two}")
    H, Hk = 4, 2
    g = torch.Generator().manual_seed(S)
    q, k = torch.zeros(1, H, T, dk, dtype=dtype, device=DEV), torch.randn(1, Hk, S, dk, generator=g).to(dtype).to(DEV)
    lam = torch.full((H,), LAM, device=DEV) if two else None
    n = (torch.arange(T) + S - T + 1) if causal else torch.full((T,), S)
    for first in range(0, S, dv):
        keys = torch.arange(first, min(first + dv, S))
        v = torch.zeros(1, Hk, S, dv, dtype=dtype, device=DEV)
        v[:, :, keys, keys - first] = 1
        o = ret.attention_fwd(q, k, v, lam, causal=causal)
        where = torch.zeros(1, 1, T, dv, dtype=torch.bool)
        where[..., :len(keys)] = keys[None] < n[:, None]
        share(o, n[None, None, :, None].double(), 1 + two, dtype, where.expand_as(o))


@pytest.mark.parametrize("two", [True, False])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dk,dv", WIDTHS)
@pytest.mark.parametrize("lens,page", [([511, 0, 1200, 33], 64), ([96, 700], 7), ([2100], 24)])
def test_step_counts_each_key(lens, page, dk, dv, dtype, two):
    say(f"each key of a step {lens} page{page} dk{dk} dv{dv} {dtype} maps={1 + two}")
    B, H, Hk = len(lens), 6, 2
    g = torch.Generator().manual_seed(page)
    table, P = pages_of(lens, page, g)
    t, n = table.to(DEV), torch.tensor(lens, dtype=I32, device=DEV)
    q, k = torch.zeros(B, H, dk, dtype=dtype, device=DEV), torch.randn(B, Hk, dk, generator=g).to(dtype).to(DEV)
    kc = torch.randn(P, Hk, page, dk, generator=g).to(dtype).to(DEV)
    lam = torch.full((H,), LAM, device=DEV) if two else None
    for first in range(0, max(lens) + 1, dv):
        rows = torch.arange(max(lens) + 1)
        one = torch.zeros(len(rows), dv)  # the value row of each token
        mine = (rows >= first) & (rows < first + dv)
        one[rows[mine], rows[mine] - first] = 1
        vc = torch.ones(P, Hk, page, dv, dtype=dtype)  # ones where no token is
        for b, m in enumerate(lens):
            s = torch.arange(m)
            vc.transpose(1, 2)[table[b, s // page].long(), s % page] = one[:m, None].to(dtype)
        v = one[torch.tensor(lens)][:, None].expand(B, Hk, dv).to(dtype).to(DEV)
        o = ret.attention_step(q, k, v, kc.clone(), vc.to(DEV), t, n, lam)
        where = torch.zeros(B, 1, dv, dtype=torch.bool)
        for b, m in enumerate(lens):
            where[b, 0, :max(0, min(dv, m + 1 - first))] = True
        share(o, (n.cpu().double() + 1)[:, None, None], 1 + two, dtype, where.expand_as(o))


def borders(n, page):
    """Keys at the borders of tiles of 32, pages and shares of 128, 256 and 512."""
    at = {0, 1, n - 1, n - 2, n // 2}
    for step in (32, 64, page, 128, 256, 512):
        at |= {m * step + d for m in range(1, n // step + 1) for d in (-1, 0)}
    return sorted(s for s in at if 0 <= s < n)


def codes(g, n, d, dtype):
    """Rows of length one in d channels, none within 0.8 of another (d > 16 random directions, or fewer keys than axes)."""
    x = torch.nn.functional.normalize(torch.randn(n, d, generator=g), dim=-1).to(dtype).float()
    near = (x @ x.T).fill_diagonal_(-1).max()
    assert near < 0.8, near
    return x


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128), (192, 96), (40, 256), (256, 256), (130, 77)])
def test_each_key_has_its_value(dk, dv, dtype):
    """A row that points at one key has that key's value: whole sequences, split keys, and steps over pages."""
    say(f"own values dk{dk} dv{dv} {dtype}")
    g = torch.Generator().manual_seed(dk)
    S, page = 1100, 24
    k = codes(g, S, dk, dtype)
    v = torch.randn(S, dv, generator=g).to(dtype)
    sharp = 200.0  # other keys' weights are below exp(-0.19 * 200): 2^-54 each

    def right(got, keys):
        want = v[keys].double()
        # the weight of all others is below 2^-43
        assert ((got.cpu().double() - want).abs() <= want.abs() * (HALF[dtype] * 1.01 + 8 * 2.0 ** -24) + 2.0 ** -40).all()

    at = torch.tensor(borders(S, page))
    kk, vv = k.to(dtype)[None, None].to(DEV), v[None, None].to(DEV)
    for some in (at, at[::40]):
        q = k[some].to(dtype)[None, None].to(DEV)
        right(ret.attention_fwd(q, kk, vv, causal=False, scale=sharp)[0, 0], some)
    # a step: a sequence for each of the keys, all of one length, the pages shared but for the last
    n = S - 1
    pages = -(-S // page)
    B = len(at)
    kc, vc = torch.zeros(pages + B, 1, page, dk, dtype=dtype), torch.zeros(pages + B, 1, page, dv, dtype=dtype)
    for s in range(n):
        kc[s // page, 0, s % page], vc[s // page, 0, s % page] = k[s].to(dtype), v[s]
    table = torch.arange(pages, dtype=I32).repeat(B, 1)
    table[:, -1] = pages + torch.arange(B, dtype=I32)
    kc[pages:], vc[pages:] = kc[pages - 1:pages].clone(), vc[pages - 1:pages].clone()
    for wide in (pages, 2000):  # 2000 pages: the keys are split for any number of sequences up to 256
        t = torch.full((B, wide), -1, dtype=I32)
        t[:, :pages] = table
        for some in (slice(None), slice(0, None, 40)):
            q = k[at[some]].to(dtype)[:, None].to(DEV)
            m = q.shape[0]
            new = [x[n].to(dtype).expand(m, 1, -1).to(DEV) for x in (k, v)]
            got = ret.attention_step(q, *new, kc.to(DEV), vc.to(DEV), t[some].contiguous().to(DEV),
                                     torch.full((m,), n, dtype=I32, device=DEV), scale=sharp)
            right(got[:, 0], at[some])


# Rounding to bf16 is off by up to 2^-8 of the value; over mantissas spread as their logarithm, by 2^-8 / sqrt(3) *
# sqrt(3 / (8 ln 2)) = 0.00166 rms.  An output has its own rounding and its weights', which move it by as much of
# itself for any spread: 0.00235; where two maps' outputs o_1 and lam o_2 cancel by a third (in square, weights of
# independent unit scores: a third of them is common), the weights' part is 0.0021: 0.0027.  A gradient has the same
# two.  A row has at most 2^-8 of either in full.  A key lost of 1200 alike moves a row by 0.029 of itself.
OUT, GRAD = 0.0032, 0.0030


def worst_row(got, want, second, lam):
    """The largest error of a row against the norms of its maps' outputs."""
    size = want.norm(dim=-1)
    if lam is not None:
        w = lam.double().view(1, -1, *[1] * (want.dim() - 2))
        size = (want + w * second).norm(dim=-1) + (w * second).norm(dim=-1)
    return float(((got.cpu().double() - want).norm(dim=-1) / size).max())


@pytest.mark.parametrize("two", [True, False])
@pytest.mark.parametrize("B,H,Hk,T,S,dk,dv,causal", [
    (1, 4, 2, 300, 300, 64, 64, True), (1, 4, 2, 511, 511, 128, 128, True), (1, 3, 3, 16, 1200, 128, 128, True),
    (1, 2, 1, 400, 400, 192, 96, False), (1, 2, 2, 333, 333, 40, 256, True), (1, 2, 1, 700, 700, 256, 256, True),
    (1, 4, 2, 257, 300, 130, 77, False)])
def test_relative_errors_in_bf16(B, H, Hk, T, S, dk, dv, causal, two):
    say(f"relative errors T{T} S{S} dk{dk} dv{dv} maps={1 + two}")
    g = torch.Generator().manual_seed(S + dk)
    q, k, v, do = (torch.randn(s, generator=g).to(BF16) for s in ((B, H, T, dk), (B, Hk, S, dk), (B, Hk, S, dv), (B, H, T, dv)))
    lam = torch.rand(H, generator=g) if two else None
    a = [None if t is None else t.to(DEV) for t in (q, k, v, lam, do)]
    o, kept = ret.attention_fwd(*a[:4], causal=causal, keep=True)
    want = oracle.attention(q, k, v, lam, causal=causal)
    assert rel_l2(o, want[0]) <= OUT and (lam is None or rel_l2(kept[1], want[2]) <= OUT)
    assert float((kept[0].cpu().double() - want[1]).abs().max()) <= 1e-4
    assert worst_row(o, want[0], want[2], lam) <= 2 * 2.0 ** -8
    grads = ret.attention_bwd(*a[:3], o, a[4], kept, a[3], causal=causal)
    for x, w in zip(grads[:3], oracle.attention_backward(q, k, v, do, lam, causal=causal)):
        assert rel_l2(x, w) <= GRAD, rel_l2(x, w)


@pytest.mark.parametrize("two", [True, False])
@pytest.mark.parametrize("lens,H,Hk,dk,dv,page", [([511, 1200], 3, 3, 40, 256, 256), ([33, 700], 4, 1, 192, 96, 64),
                                                  ([300, 0, 77], 4, 4, 256, 256, 100), ([1023, 2047], 16, 4, 128, 128, 16)])
def test_relative_errors_of_steps_in_bf16(lens, H, Hk, dk, dv, page, two):
    say(f"relative errors of steps {lens} dk{dk} dv{dv} maps={1 + two}")
    B = len(lens)
    g = torch.Generator().manual_seed(dk + page)
    table, P = pages_of(lens, page, g)
    q, k, v, kc, vc = (torch.randn(s, generator=g).to(BF16) for s in (
        (B, H, dk), (B, Hk, dk), (B, Hk, dv), (P, Hk, page, dk), (P, Hk, page, dv)))
    lam = torch.rand(H, generator=g) if two else None
    n = torch.tensor(lens, dtype=I32)
    want = oracle.attention_step(q, k, v, kc, vc, table, n, lam)[0]
    second = None if lam is None else oracle.attention_step(q[..., dk // 2:], k[..., dk // 2:], v, kc[..., dk // 2:], vc, table, n)[0]
    got = ret.attention_step(*(None if t is None else t.to(DEV) for t in (q, k, v, kc, vc, table, n, lam)))
    assert worst_row(got, want, second, lam) <= 2 * 2.0 ** -8 and rel_l2(got, want) <= OUT, rel_l2(got, want)

"""GPU parity of the gated scan (forward, backward, decode step) against the
fp64 CPU oracle, element by element.

Bounds are first-order error recursions evaluated in fp64 beside the oracle.
u = 2^-24.  c = 1 - a = -expm1(-rate softplus(-f)): the product |f| log2 e, the
exponential, the logarithm, two products and the series or difference carry at
most (32 + 2|f|) u of c.  A step of the recurrence rounds at most twice and a
value may pass a composed map instead (one more product and sum), 6 u of the
sum of magnitudes.  So the error of h obeys
    e_t = a_t e_(t-1) + u ((32 + 2|f_t|) c_t (|h|_(t-1) + |x_t|) + 6 |h|_t),
with |h| the recurrence of magnitudes; the backward recurrence likewise.
Rounding to bf16 adds 2^-8 of the value.

The hardware exponential has no subnormal results: e^-|f| below 2^-126 (|f| >
87.3) is 0, and so is a product rate e^-|f| below 2^-126.  So c and
rate sigmoid(-f) may each be off by (1 + rate) 2^-126 more (TINY below), which
df multiplies by |g| |h_(t-1) - x_t|: with values of some hundreds there the
loss reaches 1e-33, far above 2^-126 itself.
"""
import math

import pytest
import torch

import oracle
import retnet_retention_chunkwise_amd as ret
from helpers import say

pytestmark = pytest.mark.gpu

DEV, F64, U, TINY = "cuda", torch.float64, 2.0 ** -24, 2.0 ** -126
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def rates(H):
    return [2.0 ** (-4.0 * h / max(1, H - 1)) for h in range(H)]


def make(B, H, T, d, dtype, seed=0, reset=0.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(B, H, T, d, generator=g).to(dtype)
    f = (torch.randn(B, H, T, d, generator=g) * 1.5 + 2).to(dtype)
    if reset:
        f.masked_fill_(torch.rand((B, 1, T, 1), generator=g) < reset, -math.inf)
    s = torch.randn(B, H, d, generator=g)
    dy = torch.randn(B, H, T, d, generator=g).to(dtype)
    ds = torch.randn(B, H, d, generator=g)
    return x, f, s, dy, ds


def decays(f, rate):
    r = torch.tensor(rate, dtype=torch.float32).to(F64).view(1, -1, 1, 1)
    z = r * -torch.logaddexp(torch.zeros_like(f), -f)
    return torch.exp(z), -torch.expm1(z), r


def h_bounds(x, f, rate, s, normalize):
    """(|h| recurrence with |h| before every token, error bound of h), [B,H,T,d]."""
    x, f = x.to(F64), f.to(F64)
    a, c, r = decays(f, rate)
    kc = (32 + 2 * f.abs().clamp(max=1e4)) * c + (1 + r) * (TINY / U)
    ha = torch.zeros_like(x[:, :, 0]) if s is None else s.to(F64).abs()
    e = torch.zeros_like(ha)
    before, err, eb = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
    for t in range(x.shape[2]):
        ax = x[:, :, t].abs()
        before[:, :, t], eb[:, :, t] = ha, e
        hn = a[:, :, t] * ha + (c[:, :, t] * ax if normalize else ax)
        e = a[:, :, t] * e + U * (kc[:, :, t] * (ha + ax) + 6 * (hn + ha))
        ha = hn
        err[:, :, t] = e
    return before, eb, err


def g_bounds(x, f, rate, dy, s, ds, normalize):
    """Error bounds of grad_x, grad_f and grad_state_in."""
    before, eb, _ = h_bounds(x, f, rate, s, normalize)
    x, f, dy = x.to(F64), f.to(F64), dy.to(F64)
    a, c, r = decays(f, rate)
    kc = 32 + 2 * f.abs().clamp(max=1e4)
    ga = torch.zeros_like(x[:, :, 0]) if ds is None else ds.to(F64).abs()
    e = torch.zeros_like(ga)
    bx, bf = torch.empty_like(x), torch.empty_like(x)
    for t in range(x.shape[2] - 1, -1, -1):
        at, ct, kt = a[:, :, t], c[:, :, t], kc[:, :, t]
        g = dy[:, :, t].abs() + ga
        eg = e + 2 * U * g
        m = before[:, :, t] + (x[:, :, t].abs() if normalize else 0)
        k = r[:, :, 0] * torch.sigmoid(-f[:, :, t])
        tiny = (1 + r[:, :, 0]) * TINY
        bx[:, :, t] = ct * (eg + U * (kt + 1) * g) + tiny * g if normalize else eg
        bf[:, :, t] = k * (at * (eg * m + g * eb[:, :, t] + 8 * U * g * m) + (kt + 8) * U * g * m) + tiny * g * m
        e = at * eg + U * (kt * ct * g + 6 * g) + tiny * g
        ga = at * g
    return bx, bf, e


def close(name, got, want, bound, half):
    got, want = got.detach().cpu().to(F64), want.to(F64)
    lim = bound + half * want.abs() + 1e-37  # results below the smallest normal number may become 0
    worst = float(((got - want).abs() / lim).max()) if got.numel() else 0.0
    say(f"{name}: worst error {worst:.3f} of its bound")
    assert torch.isfinite(got).all() and worst <= 1.0, (name, worst)


def check_forward(name, x, f, rate, s, normalize, got_y, got_s):
    h, last = oracle.gated_scan(x, f, rate, s, normalize)
    _, _, e = h_bounds(x, f, rate, s, normalize)
    close(name + " y", got_y, h, e, HALF[x.dtype])
    if got_s is not None:
        close(name + " state", got_s, last, e[:, :, -1], U)


def check_backward(name, x, f, rate, dy, s, ds, normalize, got):
    want = oracle.gated_scan_backward(x, f, rate, dy, s, ds, normalize)
    bx, bf, bs = g_bounds(x, f, rate, dy, s, ds, normalize)
    close(name + " grad_x", got[0], want[0], bx, HALF[x.dtype])
    close(name + " grad_f", got[1], want[1], bf, HALF[x.dtype])
    if got[2] is not None:
        close(name + " grad_state", got[2], want[2], bs, U)


CASES = [
    # B, H, T, d, dtype, normalize, state, reset
    (1, 1, 1, 1, torch.float32, False, False, 0),
    (1, 2, 2, 8, torch.bfloat16, True, True, 0),
    (2, 3, 3, 5, torch.bfloat16, False, True, 0),
    (1, 1, 127, 64, torch.float32, True, True, 0),
    (1, 2, 128, 64, torch.bfloat16, False, False, 0.02),
    (2, 1, 129, 72, torch.bfloat16, True, True, 0.02),
    (1, 2, 255, 33, torch.float32, False, True, 0.1),
    (1, 3, 257, 32, torch.bfloat16, True, False, 0.01),
    (1, 1, 513, 16, torch.float32, True, True, 0.01),
    (2, 2, 600, 7, torch.bfloat16, False, True, 0.01),
    (1, 2, 1025, 130, torch.float32, False, True, 0.003),
    (1, 1, 2500, 66, torch.bfloat16, True, True, 0.001),
    (3, 5, 300, 201, torch.float32, True, False, 0.01),
    (1, 8, 700, 512, torch.bfloat16, True, True, 0.005),
    (1, 130, 140, 4, torch.float32, False, True, 0),
    (1, 1, 5000, 1, torch.float32, True, True, 0.001),
    # enough channel runs for one workgroup each
    (4, 8, 270, 512, torch.bfloat16, True, True, 0.01),
    (16, 16, 1050, 7, torch.float32, False, True, 0.01),
    # chained tiles: every access width, narrow rows, many groups
    (1, 2, 1300, 201, torch.float32, True, True, 0.003),
    (1, 1, 1500, 201, torch.bfloat16, False, True, 0.003),
    (2, 1, 2300, 24, torch.bfloat16, True, True, 0.003),
    (1, 2, 4500, 12, torch.float32, False, True, 0.003),
    (1, 130, 4300, 4, torch.bfloat16, True, True, 0.001),  # two head groups on one workspace
    (1, 1, 8000, 3, torch.float32, False, True, 0.001),
    (2, 2, 1200, 65, torch.float32, True, True, 0.003),  # one channel in the last tile
    (1, 2, 9000, 40, torch.bfloat16, False, True, 0.0005),
]


@pytest.mark.parametrize("B,H,T,d,dtype,normalize,state,reset", CASES)
def test_scan_matches_oracle(B, H, T, d, dtype, normalize, state, reset):
    name = f"scan B{B} H{H} T{T} d{d} {dtype} normalize={normalize} state={state} reset={reset}"
    say(name)
    x, f, s, dy, ds = make(B, H, T, d, dtype, seed=B + T + d, reset=reset)
    s, ds = (s, ds) if state else (None, None)
    rate = rates(H)
    X, F, DY = x.to(DEV), f.to(DEV), dy.to(DEV)
    S, DS = (s.to(DEV), ds.to(DEV)) if state else (None, None)
    y, last, kept = ret.gated_scan_fwd(X, F, rate, S, normalize=normalize, checkpoints=True)
    check_forward(name, x, f, rate, s, normalize, y, last)
    got = ret.gated_scan_bwd(X, F, rate, DY, S, DS, kept, normalize)
    check_backward(name, x, f, rate, dy, s, ds, normalize, got)
    again = ret.gated_scan_bwd(X, F, rate, DY, S, DS, None, normalize)
    assert all(torch.equal(a, b) for a, b in zip(got, again)), "checkpoints of the call and recomputed ones differ"
    assert torch.equal(X.cpu(), x) and torch.equal(DY.cpu(), dy)


@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize(
    "T,d",
    [(2, 64), (128, 39), (129, 64), (200, 66), (256, 68), (257, 39), (700, 64), (900, 65),
     (256, 32), (512, 29), (513, 32), (1700, 30), (512, 16), (1024, 13), (1025, 16), (3000, 9), (1025, 3), (3000, 2)],
)
def test_walked_bf16_runs(T, d, normalize):
    """Few blocks of tokens, on both sides of the lengths from which a run's gates are looked up."""
    H = 3
    x, f, s, dy, ds = make(2, H, T, d, torch.bfloat16, seed=7 * T + d, reset=0.004)
    f[1, 1, T // 2, d // 2] = 300.0
    f[0, 2, T - 1, 0] = -300.0
    rate = rates(H)
    y, last, kept = ret.gated_scan_fwd(x.to(DEV), f.to(DEV), rate, s.to(DEV), normalize=normalize, checkpoints=True)
    check_forward(f"walked {T} {d} {normalize}", x, f, rate, s, normalize, y, last)
    got = ret.gated_scan_bwd(x.to(DEV), f.to(DEV), rate, dy.to(DEV), s.to(DEV), ds.to(DEV), kept, normalize)
    check_backward(f"walked {T} {d} {normalize}", x, f, rate, dy, s, ds, normalize, got)


@pytest.mark.parametrize("normalize,d", [(True, 512), (False, 510)])
def test_long_bf16_sequence(normalize, d):
    """Enough chained tiles for every workgroup to look its gates up, among them gates outside the table."""
    H, T = 8, 8250
    x, f, s, dy, ds = make(1, H, T, d, torch.bfloat16, seed=31, reset=0.002)
    f[0, 3, 5000:5003, 7] = torch.tensor([300.0, -300.0, 1e-9]).bfloat16()
    rate = rates(H)
    y, last, kept = ret.gated_scan_fwd(x.to(DEV), f.to(DEV), rate, s.to(DEV), normalize=normalize, checkpoints=True)
    check_forward(f"long bf16 {normalize}", x, f, rate, s, normalize, y, last)
    got = ret.gated_scan_bwd(x.to(DEV), f.to(DEV), rate, dy.to(DEV), s.to(DEV), ds.to(DEV), kept, normalize)
    check_backward(f"long bf16 {normalize}", x, f, rate, dy, s, ds, normalize, got)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("B,H,d", [(1, 1, 1), (3, 2, 7), (8, 8, 512), (2, 130, 36)])
def test_steps_follow_the_scan(dtype, normalize, B, H, d):
    """A chain of decode steps from a state is the scan of those tokens."""
    T = 5
    name = f"step B{B} H{H} d{d} {dtype} normalize={normalize}"
    x, f, s, _, _ = make(B, H, T, d, dtype, seed=3, reset=0.2)
    state = s.to(DEV)
    X, F = x.to(DEV), f.to(DEV)
    ys = [ret.gated_scan_step(X[:, :, t].contiguous(), F[:, :, t].contiguous(), rates(H), state, normalize)
          for t in range(T)]
    check_forward(name, x, f, rates(H), s, normalize, torch.stack(ys, 2), state)
    # a token's rows taken out of the sequence by their strides
    state2 = s.to(DEV)
    ys2 = [ret.gated_scan_step(X[:, :, t], F[:, :, t], rates(H), state2, normalize) for t in range(T)]
    assert torch.equal(torch.stack(ys, 2), torch.stack(ys2, 2)) and torch.equal(state, state2)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_prefill_then_steps(dtype):
    """A prompt's final state continues in steps and in a second forward call, in place."""
    B, H, T, d = 2, 3, 300, 40
    x, f, s, _, _ = make(B, H, T, d, dtype, seed=5)
    X, F, state = x.to(DEV), f.to(DEV), s.to(DEV)
    y1, _ = ret.gated_scan_fwd(X[:, :, :200], F[:, :, :200], rates(H), state, state_out=state)
    y2, _ = ret.gated_scan_fwd(X[:, :, 200:299], F[:, :, 200:299], rates(H), state, state_out=state)
    y3 = ret.gated_scan_step(X[:, :, 299], F[:, :, 299], rates(H), state)
    check_forward("prefill, continuation, step", x, f, rates(H), s, False,
                  torch.cat([y1, y2, y3.unsqueeze(2)], 2), state)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d,T", [(64, 150), (24, 150), (19, 150), (64, 1100), (35, 1200)])
def test_strided_layouts_and_untouched_surroundings(dtype, d, T):
    """Token-major tensors and slices of fused buffers give the scan of their rows, and what lies between
    and behind the written rows stays as it was.  (Not the contiguous call's bits: narrower accesses give a
    thread more tokens, so the maps are composed in another order.)"""
    B, H, W = 2, 3, 2 * d + 5
    host = make(B, H, T, d, dtype, seed=6, reset=0.02)
    x, f, s, dy, ds = (t.to(DEV) for t in host)
    rate = rates(H)
    fused = torch.full((B, T + 3, H, W), 7.0, dtype=dtype, device=DEV)
    xs, fs = fused[:, :T, :, :d].transpose(1, 2), fused[:, :T, :, d + 3:2 * d + 3].transpose(1, 2)
    xs.copy_(x)
    fs.copy_(f)
    out = torch.full((B, T + 3, H, W), 7.0, dtype=dtype, device=DEV)
    y = out[:, :T, :, 1:d + 1].transpose(1, 2)
    got = ret.gated_scan_fwd(xs, fs, rate, s, normalize=True, y=y, checkpoints=True)
    assert got[0] is y
    check_forward(f"strided {dtype} d{d}", host[0], host[1], rate, host[2], True, got[0], got[1])
    y.fill_(7.0)
    assert torch.equal(out, torch.full_like(out, 7.0))
    gx, gf = out[:, :T, :, :d].transpose(1, 2), out[:, :T, :, d + 3:2 * d + 3].transpose(1, 2)
    dys = torch.empty(B, T, H, d, dtype=dtype, device=DEV).transpose(1, 2)
    dys.copy_(dy)
    got_g = ret.gated_scan_bwd(xs, fs, rate, dys, s, ds, got[2], True, grad_x=gx, grad_f=gf)
    check_backward(f"strided {dtype} d{d}", host[0], host[1], rate, host[3], host[2], host[4], True, got_g)
    gx.fill_(7.0)
    gf.fill_(7.0)
    assert torch.equal(out, torch.full_like(out, 7.0))
    # one sequence's inputs for a whole batch (a stride of 0)
    y0, _ = ret.gated_scan_fwd(x[:1].expand(3, H, T, d), f[:1].expand(3, H, T, d), rate, normalize=True)
    y1, _ = ret.gated_scan_fwd(x[:1], f[:1], rate, normalize=True)
    assert all(torch.equal(y0[i], y1[0]) for i in range(3))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("normalize", [False, True])
def test_extreme_gates(dtype, normalize):
    """Infinite gates, the type's largest and smallest values, tiny and huge decays and rates."""
    H, T, d = 3, 200, 16
    g = torch.Generator().manual_seed(11)
    x, _, s, dy, ds = make(1, H, T, d, dtype, seed=12)
    big = torch.finfo(dtype).max
    vals = torch.tensor([math.inf, -math.inf, big, -big, 30.0, -30.0, 90.0, -90.0, 0.0, 12.0], dtype=F64)
    f = vals[torch.randint(0, len(vals), (1, H, T, d), generator=g)].to(dtype)
    rate = [1.0, 1e-3, 40.0]
    y, last, kept = ret.gated_scan_fwd(x.to(DEV), f.to(DEV), rate, s.to(DEV), normalize=normalize, checkpoints=True)
    check_forward(f"extreme gates {dtype} {normalize}", x, f, rate, s, normalize, y, last)
    got = ret.gated_scan_bwd(x.to(DEV), f.to(DEV), rate, dy.to(DEV), s.to(DEV), ds.to(DEV), kept, normalize)
    check_backward(f"extreme gates {dtype} {normalize}", x, f, rate, dy, s, ds, normalize, got)


def test_long_memory_keeps_its_precision():
    """Constant gates with a memory of 1e5 tokens: a decay rounded to fp32 would lose 1e5 * 2^-25 = 3e-3."""
    T, d = 4000, 4
    x = torch.ones(1, 1, T, d)
    f = torch.full_like(x, 11.5)  # 1 - a = 1.01e-5
    y, last = ret.gated_scan_fwd(x.to(DEV), f.to(DEV), [1.0], normalize=True)
    h, hl = oracle.gated_scan(x, f, [1.0], None, True)
    r = float(((y.cpu().to(F64) - h) / h).abs().max())
    say(f"long memory: worst relative error {r:.2e}")
    # c: (32 + 23) u; the sum of T equal terms rounds at most once each, and here each is 2^-24 of the sum so far
    assert r <= (55 + 3 * math.sqrt(T)) * U


def test_non_finite_values_stay_in_their_channel():
    B, H, T, d = 1, 2, 300, 70
    x, f, s, _, _ = make(B, H, T, d, torch.float32, seed=13)
    clean, _ = ret.gated_scan_fwd(x.to(DEV), f.to(DEV), rates(H), s.to(DEV))
    for where, bad in (("x", math.inf), ("x", math.nan), ("f", math.nan)):
        xx, ff = x.clone(), f.clone()
        (xx if where == "x" else ff)[0, 1, 137, 66] = bad
        y, last = ret.gated_scan_fwd(xx.to(DEV), ff.to(DEV), rates(H), s.to(DEV))
        hit = torch.zeros(B, H, T, d, dtype=torch.bool, device=DEV)
        hit[0, 1, 137:, 66] = True
        assert torch.equal(y[~hit], clean[~hit]) and not torch.isfinite(y[hit]).any()
        assert not torch.isfinite(last[0, 1, 66])


def test_empty_sequence_and_optional_outputs():
    x = torch.empty(2, 3, 0, 8, device=DEV)
    s = torch.randn(2, 3, 8, device=DEV)
    y, last = ret.gated_scan_fwd(x, x, rates(3), s)
    assert y.shape == x.shape and torch.equal(last, s)
    assert torch.equal(ret.gated_scan_fwd(x, x, rates(3))[1], torch.zeros_like(s))
    gx, gf, gs = ret.gated_scan_bwd(x, x, rates(3), x, s, s)
    assert gx.shape == x.shape and gf.shape == x.shape and torch.equal(gs, s)
    x, f, s0, dy, _ = (t.to(DEV) for t in make(2, 3, 20, 8, torch.bfloat16))
    y, last = ret.gated_scan_fwd(x, f, rates(3), s0, state_out=False)
    assert last is None and torch.equal(y, ret.gated_scan_fwd(x, f, rates(3), s0)[0])
    a, b = ret.gated_scan_bwd(x, f, rates(3), dy, s0, grad_state_in=False), ret.gated_scan_bwd(x, f, rates(3), dy, s0)
    assert a[2] is None and torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_grad_state_in_place():
    x, f, s, dy, ds = (t.to(DEV) for t in make(2, 3, 150, 40, torch.float32))
    want = ret.gated_scan_bwd(x, f, rates(3), dy, s, ds)[2]
    buf = ds.clone()
    got = ret.gated_scan_bwd(x, f, rates(3), dy, s, buf, grad_state_in=buf)[2]
    assert got is buf and torch.equal(buf, want)


@pytest.mark.parametrize("B,H,T,d", [(1, 2, 3000, 64), (4, 8, 300, 512)])
def test_graph_replays_and_other_streams(B, H, T, d):
    """Forward and backward captured together: every replay, with eager calls of other sizes in between,
    matches the eager call bit for bit; so does a call on another stream."""
    x, f, s, dy, ds = (t.to(DEV) for t in make(B, H, T, d, torch.bfloat16, seed=21, reset=0.01))
    rate = rates(H)

    def step():
        y, last, kept = ret.gated_scan_fwd(x, f, rate, s, normalize=True, checkpoints=True)
        return (y, last, *ret.gated_scan_bwd(x, f, rate, dy, s, ds, kept, True))

    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(other, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for i in range(4):
        for t in got:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i
        ret.gated_scan_fwd(x[:, :, : T // 2], f[:, :, : T // 2], rate)
        torch.cuda.synchronize()


@pytest.mark.parametrize("B,H,T,d,dtype", [(2, 4, 1500, 64, torch.bfloat16), (3, 5, 1337, 201, torch.float32)])
def test_other_inputs_on_the_same_workspace(B, H, T, d, dtype):
    """Calls of different inputs one after the other, on workspaces that hold the last call's words: each
    gives the bits it gives alone.  A call over another call's inputs in a captured graph too."""
    rate = rates(H)
    sets = [[t.to(DEV) for t in make(B, H, T, d, dtype, seed=60 + i, reset=0.003)] for i in range(3)]
    lib = ret.load()
    fb = lib.retention_gated_scan_workspace_bytes(B, H, T, d, 1)
    bb = lib.retention_gated_scan_bwd_workspace_bytes(B, H, T, d, 1, 1)
    assert fb > 0 and bb > 0
    ws, wb = (torch.full((n,), 0xA5, dtype=torch.uint8, device=DEV) for n in (fb, bb))

    def step(v):
        x, f, s, dy, ds = v
        y, last, kept = ret.gated_scan_fwd(x, f, rate, s, normalize=True, checkpoints=True, workspace=ws)
        return [y, last, *ret.gated_scan_bwd(x, f, rate, dy, s, ds, kept, True, workspace=wb)]

    alone = []
    for v in sets:
        alone.append([t.clone() for t in step(v)])
        torch.cuda.synchronize()
    for _ in range(5):
        got = [step(v) for v in sets]
        torch.cuda.synchronize()
        for g, a in zip(got, alone):
            assert all(torch.equal(p, q) for p, q in zip(g, a))
    held = [t.clone() for t in sets[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(held)
    for i in (1, 2, 0, 1):
        for t, v in zip(held, sets[i]):
            t.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(out, alone[i])), i
        step(sets[(i + 1) % 3])


def test_binding_refuses():
    x, f, s, dy, _ = (t.to(DEV) for t in make(1, 2, 20, 8, torch.float32))
    r = rates(2)
    for bad in (lambda: ret.gated_scan_fwd(x, f.bfloat16(), r), lambda: ret.gated_scan_fwd(x, f[:, :, :10], r),
                lambda: ret.gated_scan_fwd(x.half(), f.half(), r), lambda: ret.gated_scan_fwd(x, f, [1.0]),
                lambda: ret.gated_scan_fwd(x.transpose(2, 3), f.transpose(2, 3), r),
                lambda: ret.gated_scan_fwd(x, f, r, s.bfloat16()), lambda: ret.gated_scan_fwd(x.cpu(), f.cpu(), r),
                lambda: ret.gated_scan_fwd(x, f, r, y=x), lambda: ret.gated_scan_fwd(x, f, [1.0, -1.0]),
                lambda: ret.gated_scan_bwd(x, f, r, dy, grad_x=x), lambda: ret.gated_scan_bwd(x, f, r, dy[:, :, :3]),
                lambda: ret.gated_scan_bwd(x, f, r, dy, checkpoints=s), lambda: ret.gated_scan_step(x[:, :, 0], f[:, :, 0], r, None),
                lambda: ret.gated_scan_fwd(x, f, r, y=x[:, :, :1].expand(1, 2, 20, 8))):
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            bad()

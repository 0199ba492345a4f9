"""Refusals of the block operators' C entry points (no GPU: every call below
fails validation before any HIP call)."""
import ctypes

import pytest

from retnet_retention_chunkwise_amd import _lib

INVALID, UNSUPPORTED = _lib.RET_ERR_INVALID_ARG, _lib.RET_ERR_UNSUPPORTED
BAD = ctypes.c_size_t(-1).value


def at(n, off=0):
    """A made-up address, never dereferenced, far from the others."""
    return ctypes.c_void_p((n << 36) + off)


def fl(*v):
    return (ctypes.c_float * len(v))(*v)


def st(*rows):
    flat = [x for r in rows for x in r]
    return (ctypes.c_longlong * len(flat))(*flat)


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def scan_fwd(lib, x=at(1), f=at(2), rate=fl(1.0, 0.5), sin=None, sout=None, y=at(3), ck=None, strides=None, B=1, H=2,
             T=8, d=16, norm=0, dt=0, ws=None, wsb=0):
    return lib.retention_gated_scan_fwd(x, f, rate, sin, sout, y, ck, strides, B, H, T, d, norm, dt, ws, wsb, None)


C = (256, 128, 16)  # contiguous strides of [1,2,8,16]


@pytest.mark.parametrize("kw,status,needle", [
    (dict(B=0), INVALID, "B=0"),
    (dict(H=0), INVALID, "H=0"),
    (dict(T=-1), INVALID, "T=-1"),
    (dict(d=0), INVALID, "d=0"),
    (dict(dt=3), UNSUPPORTED, "dtype"),
    (dict(T=(1 << 30) + 1, d=1, H=1, rate=fl(1.0)), UNSUPPORTED, "2^30"),
    (dict(B=1 << 10, T=1 << 20), UNSUPPORTED, "2^31"),
    (dict(B=1 << 30, H=1 << 30, rate=fl(1.0)), UNSUPPORTED, "2^31"),
    (dict(B=(1 << 21) + 1, H=1, T=2, rate=fl(1.0)), UNSUPPORTED, "2^21"),
    (dict(rate=None), INVALID, "rate"),
    (dict(rate=fl(1.0, 0.0)), INVALID, "rate[1]"),
    (dict(rate=fl(-1.0, 1.0)), INVALID, "rate[0]"),
    (dict(rate=fl(1.0, float("inf"))), INVALID, "rate[1]"),
    (dict(rate=fl(float("nan"), 1.0)), INVALID, "rate[0]"),
    (dict(x=None), INVALID, "x is required"),
    (dict(f=None), INVALID, "f is required"),
    (dict(y=None), INVALID, "y is required"),
    (dict(x=at(1, 2)), UNSUPPORTED, "aligned"),
    (dict(dt=1, y=at(3, 1)), UNSUPPORTED, "aligned"),
    (dict(sin=at(4, 4)), UNSUPPORTED, "state_in must be aligned"),
    (dict(ck=at(4, 8)), UNSUPPORTED, "checkpoints must be aligned"),
    (dict(y=at(1)), INVALID, "overlaps"),
    (dict(y=at(2, 256 * 4 - 4)), INVALID, "y overlaps f"),
    (dict(sin=at(4), sout=at(4, 16)), INVALID, "overlaps"),
    (dict(sout=at(3)), INVALID, "overlaps"),
    (dict(ck=at(1)), INVALID, "overlaps"),
    (dict(strides=st(C, C, (256, -128, 16))), INVALID, "stride"),
    (dict(strides=st(C, (256, 1 << 47, 16), C)), INVALID, "stride"),
    (dict(strides=st(C, C, (256, 128, 15))), INVALID, "rows of y overlap"),
    (dict(strides=st(C, C, (256, 0, 16))), INVALID, "rows of y overlap"),
    (dict(strides=st(C, C, (256, 112, 16))), INVALID, "rows of y overlap"),
    # slices of one buffer of 32-element rows: y's columns 8..23 meet x's 0..15
    (dict(y=at(1, 32), strides=st((512, 256, 32), C, (512, 256, 32))), INVALID, "y overlaps x"),
])
def test_scan_forward_refuses(lib, kw, status, needle):
    assert scan_fwd(lib, **kw) == status
    assert needle in _lib.last_error(), _lib.last_error()


def test_interleaved_slices_are_told_from_overlaps(lib):
    """Slices that only interleave pass the overlap checks: the refusal is the one planted behind them."""
    s = (512, 256, 32)
    kw = dict(y=at(1, 64), strides=st(s, C, s), sin=at(1, 64), sout=at(1, 64 + 16))
    assert scan_fwd(lib, **kw) == INVALID and "y overlaps state" in _lib.last_error()
    kw = dict(y=at(1, 64), strides=st(s, C, s), sin=at(5), sout=at(5, 16))
    assert scan_fwd(lib, **kw) == INVALID and "state_out" in _lib.last_error()


def scan_bwd(lib, x=at(1), f=at(2), rate=fl(1.0, 0.5), sin=None, ck=at(7), gy=at(3), gso=None, gx=at(4), gf=at(5),
             gsi=None, strides=None, B=1, H=2, T=8, d=16, norm=0, dt=0, ws=None, wsb=0):
    return lib.retention_gated_scan_bwd(x, f, rate, sin, ck, gy, gso, gx, gf, gsi, strides, B, H, T, d, norm, dt, ws,
                                        wsb, None)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(H=0), INVALID, "H=0"),
    (dict(rate=fl(1.0, -0.5)), INVALID, "rate[1]"),
    (dict(gy=None), INVALID, "grad_y is required"),
    (dict(gx=None), INVALID, "grad_x is required"),
    (dict(gf=None), INVALID, "grad_f is required"),
    (dict(gx=at(1)), INVALID, "overlaps"),
    (dict(gf=at(4)), INVALID, "overlaps"),
    (dict(gsi=at(7)), INVALID, "overlaps"),
    (dict(gso=at(8), gsi=at(8, 16)), INVALID, "overlaps"),
    (dict(ck=at(4)), INVALID, "overlaps"),
    (dict(ck=None), INVALID, "workspace"),
    (dict(ck=None, ws=at(9), wsb=4), INVALID, "workspace"),
    (dict(ck=None, ws=at(5), wsb=1 << 20), INVALID, "overlaps"),
    (dict(ck=None, ws=at(9, 4), wsb=1 << 20), UNSUPPORTED, "workspace must be aligned"),
])
def test_scan_backward_refuses(lib, kw, status, needle):
    assert scan_bwd(lib, **kw) == status
    assert needle in _lib.last_error(), _lib.last_error()


def test_scan_step_refuses(lib):
    call = lambda x=at(1), f=at(2), s=at(3), y=at(4), d=16, dt=0: lib.retention_gated_scan_step(  # noqa: E731
        x, f, fl(1.0), s, y, None, 1, 1, d, 0, dt, None)
    assert call(s=None) == INVALID and "state is required" in _lib.last_error()
    assert call(y=at(3)) == INVALID and "overlaps" in _lib.last_error()
    assert call(y=at(1)) == INVALID and "overlaps" in _lib.last_error()
    assert call(s=at(3, 4)) == UNSUPPORTED and "aligned" in _lib.last_error()
    assert call(d=0) == INVALID


def test_scan_sizes(lib):
    assert lib.retention_gated_scan_workspace_bytes(0, 1, 1, 1, 0) == BAD
    assert lib.retention_gated_scan_checkpoint_bytes(1, 1, -1, 1) == BAD
    assert lib.retention_gated_scan_bwd_workspace_bytes(1, 1, 1, 0, 0, 0) == BAD
    assert lib.retention_gated_scan_checkpoint_bytes(2, 3, 0, 64) == 0
    one = lib.retention_gated_scan_checkpoint_bytes(2, 3, 1, 64)
    assert one == 2 * 3 * 64 * 4  # one block, whatever its length
    assert lib.retention_gated_scan_bwd_workspace_bytes(2, 3, 1, 64, 0, 0) >= one


# ------------------------------------------------------------------- norms
def gn(lib, y=at(1), z=at(2), w=None, b=None, eps=1e-5, out=at(3), strides=None, B=2, H=2, T=4, dv=16, dt=0):
    return lib.retention_group_norm_gated(y, z, w, b, eps, out, strides, B, H, T, dv, dt, None)


def gnb(lib, y=at(1), z=at(2), w=at(8), b=None, eps=1e-5, do=at(3), gy=at(4), gz=at(5), gw=at(9), gb=None,
        strides=None, B=2, H=2, T=4, dv=16, dt=0, ws=None, wsb=0):
    return lib.retention_group_norm_gated_bwd(y, z, w, b, eps, do, gy, gz, gw, gb, strides, B, H, T, dv, dt, ws, wsb,
                                              None)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(B=0), INVALID, "B=0"),
    (dict(dv=513), UNSUPPORTED, "513"),
    (dict(H=65536), UNSUPPORTED, "65536"),
    (dict(T=1 << 28, dv=1), UNSUPPORTED, "2^28"),
    (dict(dt=2), UNSUPPORTED, "dtype"),
    (dict(eps=-1e-5), INVALID, "eps"),
    (dict(eps=float("nan")), INVALID, "eps"),
    (dict(y=None), INVALID, "y is required"),
    (dict(out=None), INVALID, "out is required"),
    (dict(out=at(1)), INVALID, "overlaps"),
    (dict(out=at(2)), INVALID, "overlaps"),
    (dict(w=at(3)), INVALID, "overlaps"),
    (dict(b=at(8, 4)), UNSUPPORTED, "bias must be aligned"),
    (dict(strides=st((128, 64, 16), (128, 16, 32), (128, 15, 32))), INVALID, "rows of out overlap"),
])
def test_gate_norm_refuses(lib, kw, status, needle):
    assert gn(lib, **kw) == status
    assert needle in _lib.last_error(), _lib.last_error()


@pytest.mark.parametrize("kw,status,needle", [
    (dict(T=-1), INVALID, "T=-1"),
    (dict(dv=513), UNSUPPORTED, "513"),
    (dict(z=None), INVALID, "together"),
    (dict(gz=None), INVALID, "together"),
    (dict(do=None), INVALID, "grad_out is required"),
    (dict(gy=None), INVALID, "grad_y is required"),
    (dict(gy=at(3)), INVALID, "overlaps"),
    (dict(gz=at(4)), INVALID, "overlaps"),
    (dict(gw=at(8)), INVALID, "overlaps"),
    (dict(), INVALID, "workspace"),
    (dict(ws=at(10), wsb=16), INVALID, "workspace"),
    (dict(ws=at(4), wsb=1 << 24), INVALID, "overlaps"),
])
def test_gate_norm_backward_refuses(lib, kw, status, needle):
    assert gnb(lib, **kw) == status
    assert needle in _lib.last_error(), _lib.last_error()


def rn(lib, x=at(1), f=at(2), w=None, b=None, s=None, alpha=1.0, eps=1e-5, r=at(3), n=at(4), strides=None, rows=8,
       D=16, dt=0):
    return lib.retention_residual_norm(x, f, w, b, s, alpha, eps, 0, r, n, strides, rows, D, dt, None)


def rnb(lib, r=at(1), dn=at(2), dr=None, f=None, w=None, s=None, alpha=1.0, eps=1e-5, gx=at(3), gf=at(4), gw=None,
        gb=None, gs=None, strides=None, rows=8, D=16, dt=0, ws=None, wsb=0):
    return lib.retention_residual_norm_bwd(r, dn, dr, f, w, s, alpha, eps, 0, gx, gf, gw, gb, gs, strides, rows, D, dt,
                                           ws, wsb, None)


def ll(*v):
    return (ctypes.c_longlong * len(v))(*v)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(rows=-1), INVALID, "rows=-1"),
    (dict(D=0), INVALID, "D=0"),
    (dict(D=16385), UNSUPPORTED, "16385"),
    (dict(rows=(1 << 28) + 1, D=1), UNSUPPORTED, "2^28"),
    (dict(rows=1 << 20, D=4096), UNSUPPORTED, "2^31"),
    (dict(alpha=float("inf")), INVALID, "alpha"),
    (dict(eps=-1.0), INVALID, "eps"),
    (dict(f=None), INVALID, "f is required"),
    (dict(n=None), INVALID, "n is required"),
    (dict(r=at(1)), INVALID, "overlaps"),
    (dict(n=at(3)), INVALID, "overlaps"),
    (dict(s=at(6, 8)), UNSUPPORTED, "aligned"),
    (dict(strides=ll(16, 16, 8, 16)), INVALID, "rows of r overlap"),
    (dict(strides=ll(16, -16, 16, 16)), INVALID, "stride"),
])
def test_residual_norm_refuses(lib, kw, status, needle):
    assert rn(lib, **kw) == status
    assert needle in _lib.last_error(), _lib.last_error()


@pytest.mark.parametrize("kw,status,needle", [
    (dict(r=None), INVALID, "r is required"),
    (dict(dn=None), INVALID, "grad_n is required"),
    (dict(gs=at(7), ws=at(9), wsb=1 << 24), INVALID, "f is required"),
    (dict(gx=at(1)), INVALID, "overlaps"),
    (dict(gf=at(3)), INVALID, "overlaps"),
    (dict(gw=at(7), gb=at(7), ws=at(9), wsb=1 << 24), INVALID, "overlaps"),
    (dict(gw=at(7)), INVALID, "workspace"),
    (dict(gw=at(7), ws=at(9, 8), wsb=1 << 24), UNSUPPORTED, "aligned"),
])
def test_residual_norm_backward_refuses(lib, kw, status, needle):
    assert rnb(lib, **kw) == status
    assert needle in _lib.last_error(), _lib.last_error()


def test_norm_sizes(lib):
    assert lib.retention_group_norm_gated_bwd_workspace_bytes(1, 1, 1, 513) == BAD
    assert lib.retention_group_norm_gated_bwd_workspace_bytes(1, 1, 0, 8) == 0
    assert lib.retention_group_norm_gated_bwd_workspace_bytes(2, 3, 1, 8) == 2 * 1 * 3 * 8 * 4
    assert lib.retention_residual_norm_bwd_workspace_bytes(-1, 8) == BAD
    assert lib.retention_residual_norm_bwd_workspace_bytes(0, 8) == 0
    assert lib.retention_residual_norm_bwd_workspace_bytes(1, 8) == 3 * 8 * 4


def test_merged_heads_of_one_buffer(lib):
    """[B,T,H*dv] slices of a fused buffer interleave by tokens: disjoint columns pass, meeting ones do not."""
    W, row = 2 * 16, 2 * 32 + 5  # two heads of 16; token rows of 69 elements
    y, t = (128, 64, 16), (4 * row, 16, row)
    kw = dict(strides=st(y, t, t, (4 * row, 16, row), t), do=at(5, 4 * 0), z=at(2), gz=at(4, 4 * W), gy=at(4, 4 * 0))
    assert gnb(lib, **kw) == INVALID and "workspace" in _lib.last_error(), _lib.last_error()
    kw["gz"] = at(4, 4 * (W - 1))
    assert gnb(lib, **kw) == INVALID and "overlaps" in _lib.last_error(), _lib.last_error()
    kw["gz"] = at(4, 4 * (row - W))  # ends where the next token's row of grad_y begins
    assert gnb(lib, **kw) == INVALID and "workspace" in _lib.last_error(), _lib.last_error()
    kw["gz"] = at(4, 4 * (row - W + 1))
    assert gnb(lib, **kw) == INVALID and "overlaps" in _lib.last_error(), _lib.last_error()

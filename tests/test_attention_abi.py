"""Refusals of the attention calls' C entry points (no GPU: every call below
fails validation before any HIP call), and their workspace sizes."""
import ctypes

import pytest
import torch

import retnet_retention_chunkwise_amd as ret
from retnet_retention_chunkwise_amd import _lib

INVALID, UNSUPPORTED = _lib.RET_ERR_INVALID_ARG, _lib.RET_ERR_UNSUPPORTED
BAD = ctypes.c_size_t(-1).value


def at(n, off=0):
    """A made-up address, never dereferenced, far from the others."""
    return ctypes.c_void_p((n << 40) + off)


def st(*rows):
    flat = [x for r in rows for x in r]
    return (ctypes.c_longlong * len(flat))(*flat)


@pytest.fixture(scope="module")
def lib():
    return _lib.load()


def fwd(lib, q=at(1), k=at(2), v=at(3), lam=at(4), lens=None, o=at(5), lse=None, second=None, strides=None, B=1, H=4, Hk=2,
        T=8, S=8, dk=16, dv=16, scale=0.25, causal=1, offset=0, dt=0, ws=None, wsb=0):
    return lib.retention_attention_fwd(q, k, v, lam, lens, o, lse, second, strides, B, H, Hk, T, S, dk, dv, scale, causal,
                                       offset, dt, ws, wsb, None)


Q, K = (512, 128, 16), (256, 128, 16)  # contiguous strides of [1,4,8,16] and [1,2,8,16]
SIZES = [
    (dict(B=0), INVALID, "B=0"),
    (dict(H=0), INVALID, "H=0"),
    (dict(Hk=0), INVALID, "Hk=0"),
    (dict(Hk=3), INVALID, "multiple of Hk=3"),
    (dict(T=-1), INVALID, "T=-1"),
    (dict(S=-1), INVALID, "S=-1"),
    (dict(dk=0), INVALID, "dk=0"),
    (dict(dv=0), INVALID, "dv=0"),
    (dict(dk=17), INVALID, "halve"),
    (dict(dk=258), UNSUPPORTED, "258"),
    (dict(dv=257), UNSUPPORTED, "257"),
    (dict(dt=2), UNSUPPORTED, "dtype"),
    (dict(T=(1 << 30) + 1), UNSUPPORTED, "2^30"),
    (dict(T=1 << 25), UNSUPPORTED, "2^31"),
    (dict(B=1 << 30, H=1 << 30, Hk=1), UNSUPPORTED, "2^31"),
    (dict(B=1 << 12, T=1 << 12, dk=2, dv=1), UNSUPPORTED, "2^25"),
    (dict(B=1 << 22, Hk=4, T=1, S=1, dk=2, dv=2), UNSUPPORTED, "2^23"),
    (dict(scale=0.0), INVALID, "scale"),
    (dict(scale=-1.0), INVALID, "scale"),
    (dict(scale=float("inf")), INVALID, "scale"),
    (dict(scale=float("nan")), INVALID, "scale"),
    (dict(offset=(1 << 30) + 1), INVALID, "offset"),
    (dict(offset=-(1 << 30) - 1), INVALID, "offset"),
    (dict(q=None), INVALID, "q is required"),
    (dict(k=None), INVALID, "k is required"),
    (dict(v=None), INVALID, "v is required"),
    (dict(o=None), INVALID, "o is required"),
    (dict(q=at(1, 2)), UNSUPPORTED, "aligned"),
    (dict(dt=1, v=at(3, 1)), UNSUPPORTED, "aligned"),
    (dict(lam=at(4, 2)), UNSUPPORTED, "lam must be aligned"),
    (dict(lens=at(6, 1)), UNSUPPORTED, "lens must be aligned"),
]


@pytest.mark.parametrize("kw,status,needle", SIZES + [
    (dict(lam=None, second=at(7)), INVALID, "second"),
    (dict(o=at(1)), INVALID, "o overlaps q"),
    (dict(o=at(2, 256 * 4 - 4)), INVALID, "o overlaps k"),
    (dict(o=at(4)), INVALID, "overlaps"),
    (dict(lse=at(5, 2048 - 4)), INVALID, "o overlaps lse"),
    (dict(second=at(5)), INVALID, "o overlaps second"),
    (dict(strides=st(Q, K, K, (512, 128, 15))), INVALID, "rows of o overlap"),
    (dict(strides=st(Q, K, K, (512, 0, 16))), INVALID, "rows of o overlap"),
    (dict(strides=st(Q, (256, -128, 16), K, Q)), INVALID, "stride"),
    (dict(strides=st(Q, (1 << 28, 16, (1 << 24) + 1), K, Q)), UNSUPPORTED, "2^24"),
    (dict(strides=st(Q, K, (256, 1 << 47, 16), Q)), INVALID, "stride"),
    (dict(S=4096), INVALID, "workspace"),
    (dict(S=4096, ws=at(9), wsb=64), INVALID, "workspace"),
    (dict(S=4096, ws=at(9, 8), wsb=1 << 30), UNSUPPORTED, "workspace must be aligned"),
    (dict(S=4096, ws=at(5), wsb=1 << 30), INVALID, "overlaps"),
])
def test_forward_refuses(lib, kw, status, needle):
    assert fwd(lib, **kw) == status
    assert needle in _lib.last_error(), _lib.last_error()


def bwd(lib, q=at(1), k=at(2), v=at(3), lam=at(4), lens=None, o=at(5), lse=at(6), second=at(7), go=at(8), gq=at(9), gk=at(10),
        gv=at(11), gl=at(12), strides=None, B=1, H=4, Hk=2, T=8, S=8, dk=16, dv=16, scale=0.25, causal=1, offset=0, dt=0,
        ws=at(13), wsb=1 << 20):
    return lib.retention_attention_bwd(q, k, v, lam, lens, o, lse, second, go, gq, gk, gv, gl, strides, B, H, Hk, T, S, dk, dv,
                                       scale, causal, offset, dt, ws, wsb, None)


@pytest.mark.parametrize("kw,status,needle", [c for c in SIZES if not set(c[0]) & {"lens"}] + [
    (dict(lse=None), INVALID, "lse is required"),
    (dict(second=None), INVALID, "second is required"),
    (dict(lam=None), INVALID, "together"),
    (dict(gl=None), INVALID, "together"),
    (dict(go=None), INVALID, "grad_o is required"),
    (dict(gq=None), INVALID, "grad_q is required"),
    (dict(gk=None), INVALID, "grad_k is required"),
    (dict(gv=None), INVALID, "grad_v is required"),
    (dict(gq=at(1)), INVALID, "overlaps"),
    (dict(gk=at(9)), INVALID, "overlaps"),
    (dict(gv=at(3)), INVALID, "overlaps"),
    (dict(gl=at(6, 16)), INVALID, "overlaps"),
    (dict(gq=at(7)), INVALID, "overlaps"),
    (dict(strides=st((1 << 28, 16, 1 << 25), K, K, Q, Q, Q, K, K)), UNSUPPORTED, "2^24"),
    (dict(ws=None), INVALID, "workspace"),
    (dict(wsb=8), INVALID, "workspace"),
    (dict(ws=at(13, 4)), UNSUPPORTED, "aligned"),
    (dict(ws=at(8)), INVALID, "overlaps"),
])
def test_backward_refuses(lib, kw, status, needle):
    assert bwd(lib, **kw) == status
    assert needle in _lib.last_error(), _lib.last_error()


def step(lib, q=at(1), k=at(2), v=at(3), kc=at(4), vc=at(5), table=at(6), lens=at(7), lam=None, o=at(8), strides=None, B=2,
         H=4, Hk=2, dk=16, dv=16, pages=8, page=4, most=3, scale=0.25, dt=0, ws=None, wsb=0):
    return lib.retention_attention_step(q, k, v, kc, vc, table, lens, lam, o, strides, B, H, Hk, dk, dv, pages, page, most,
                                        scale, dt, ws, wsb, None)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(B=0), INVALID, "B=0"),
    (dict(Hk=3), INVALID, "multiple"),
    (dict(dk=15, lam=at(9)), INVALID, "halve"),
    (dict(dk=257), UNSUPPORTED, "257"),
    (dict(dt=7), UNSUPPORTED, "dtype"),
    (dict(pages=-1), INVALID, "pages=-1"),
    (dict(page=0), INVALID, "page=0"),
    (dict(most=-1), INVALID, "max_pages=-1"),
    (dict(page=1 << 16, most=1 << 15), UNSUPPORTED, "2^30"),
    (dict(B=1 << 23), UNSUPPORTED, "2^23"),
    (dict(scale=0.0), INVALID, "scale"),
    (dict(q=None), INVALID, "q is required"),
    (dict(k=None), INVALID, "k is required"),
    (dict(kc=None), INVALID, "k_cache is required"),
    (dict(vc=None), INVALID, "v_cache is required"),
    (dict(table=None), INVALID, "table is required"),
    (dict(lens=None), INVALID, "lens is required"),
    (dict(o=None), INVALID, "o is required"),
    (dict(table=at(6, 2)), UNSUPPORTED, "aligned"),
    (dict(vc=at(4)), INVALID, "overlaps"),
    (dict(o=at(4, 64)), INVALID, "overlaps"),
    (dict(k=at(4, 64)), INVALID, "overlaps"),
    (dict(o=at(1)), INVALID, "overlaps"),
    (dict(strides=st((64, 16, 0), (32, 16, 0), (32, 16, 0), (128, 64, 8), (128, 64, 16), (64, 16, 0))), INVALID,
     "rows of k_cache overlap"),
    (dict(page=256, most=64), INVALID, "workspace"),
    (dict(page=256, most=64, ws=at(9), wsb=128), INVALID, "workspace"),
    (dict(page=256, most=64, ws=at(4), wsb=1 << 30), INVALID, "overlaps"),
])
def test_step_refuses(lib, kw, status, needle):
    assert step(lib, **kw) == status
    assert needle in _lib.last_error(), _lib.last_error()


def append(lib, k=at(2), v=at(3), kc=at(4), vc=at(5), table=at(6), start=at(7), counts=None, strides=None, B=2, Hk=2, T=5,
           dk=16, dv=16, pages=8, page=4, most=3, dt=0):
    return lib.retention_cache_append(k, v, kc, vc, table, start, counts, strides, B, Hk, T, dk, dv, pages, page, most, dt,
                                      None)


@pytest.mark.parametrize("kw,status,needle", [
    (dict(B=0), INVALID, "B=0"),
    (dict(T=-1), INVALID, "T=-1"),
    (dict(dv=300), UNSUPPORTED, "300"),
    (dict(page=0), INVALID, "page=0"),
    (dict(page=1 << 20, most=1 << 20), UNSUPPORTED, "2^30"),
    (dict(k=None), INVALID, "k is required"),
    (dict(kc=None), INVALID, "k_cache is required"),
    (dict(table=None), INVALID, "table is required"),
    (dict(start=None), INVALID, "start is required"),
    (dict(counts=at(8, 3)), UNSUPPORTED, "counts must be aligned"),
    (dict(kc=at(2)), INVALID, "overlaps"),
    (dict(vc=at(4, 16)), INVALID, "overlaps"),
])
def test_append_refuses(lib, kw, status, needle):
    assert append(lib, **kw) == status
    assert needle in _lib.last_error(), _lib.last_error()


def test_calls_without_work_reach_no_device(lib):
    """No rows, or no cache to store to: accepted and done, without a GPU here."""
    assert fwd(lib, T=0) == 0 and fwd(lib, T=0, q=None, o=None) == 0
    assert append(lib, T=0) == 0 and append(lib, most=0, table=None) == 0 and append(lib, pages=0, kc=None, vc=None) == 0


def test_sizes(lib):
    size = lib.retention_attention_workspace_bytes
    assert size(1, 4, 3, 8, 8, 16, 16, 1, 0) == BAD and "multiple" in _lib.last_error()
    assert size(1, 4, 2, 8, 8, 16, 16, 3, 0) == BAD and "maps=3" in _lib.last_error()
    assert size(1, 4, 2, 0, 1 << 20, 16, 16, 1, 0) == 0
    assert size(8, 16, 16, 4096, 4096, 64, 64, 2, 1) == 0  # rows enough to fill the device
    assert size(1, 4, 2, 1, 8192, 64, 64, 2, 1) > 0
    size = lib.retention_attention_bwd_workspace_bytes
    assert size(1, 4, 2, 8, 8, 17, 16, 2, 0) == BAD
    assert size(1, 4, 2, 8, 8, 16, 16, 1, 0) >= 4 * 8 * 8 and size(1, 4, 2, 8, 8, 16, 16, 2, 0) > size(1, 4, 2, 8, 8, 16, 16, 1, 0)
    size = lib.retention_attention_step_workspace_bytes
    assert size(1, 4, 2, 16, 16, 0, 8, 1, 0) == BAD and size(1 << 23, 4, 2, 16, 16, 4, 8, 1, 0) == BAD
    assert size(1, 4, 2, 16, 16, 16, 4, 1, 0) == 0 and size(1, 4, 2, 16, 16, 16, 4096, 2, 1) > 0


def test_binding_refuses():
    """What the binding tells before the library is asked (tensors on the CPU)."""
    t = torch.zeros
    q, k, v = t(1, 4, 8, 16), t(1, 2, 8, 16), t(1, 2, 8, 16)
    for call in (lambda: ret.attention_fwd(q, k, v), lambda: ret.attention_step(q[:, :, 0], k[:, :, 0], v[:, :, 0], k, v, None, None),
                 lambda: ret.cache_append(k, v, k, v, None, None)):
        with pytest.raises(ValueError, match="device"):
            call()
    with pytest.raises(ValueError, match="expected q"):
        ret.attention_fwd(q[0], k, v)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        ret.attention_fwd(q.half(), k.half(), v.half())
    with pytest.raises(ValueError, match="expected q"):
        ret.attention_step(q, k, v, k, v, None, None)
    with pytest.raises(ValueError, match="expected k"):
        ret.cache_append(k[0], v[0], k, v, None, None)

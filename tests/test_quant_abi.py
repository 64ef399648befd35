"""CPU checks of the norm, quantiser and 8-bit product entry points: bad
arguments are refused before any HIP call."""
import ctypes
import math

import pytest

import selective_state_space_80_amd as mamba

F32, BF16 = mamba.MAMBA_F32, mamba.MAMBA_BF16
OK, ENULL, ESHAPE, EDTYPE, EUNSUP, EALIGN, EALIAS, EWS, ELAUNCH, EDEV, ETIMEOUT = range(11)


@pytest.fixture(scope="module")
def lib():
    return mamba.load_library()


def _p(k):
    """Made-up device addresses, far apart: never dereferenced on the host."""
    return ctypes.c_void_p(k << 40)


X, R, W, O, RO, S, WS, DX, DR = (_p(k) for k in range(1, 10))


def norm(lib, **kw):
    a = dict(x=X, residual=R, weight=W, out=O, residual_out=RO, M=4, D=64, eps=1e-5, io=BF16, rt=F32, stream=None)
    a.update(kw)
    return lib.mamba_rms_norm(*a.values())


def norm8(lib, **kw):
    a = dict(x=X, residual=R, weight=W, out=O, scale=S, residual_out=RO, M=4, D=64, eps=1e-5, io=BF16, rt=F32,
             stream=None)
    a.update(kw)
    return lib.mamba_rms_norm_int8(*a.values())


@pytest.mark.parametrize("call", [norm, norm8])
@pytest.mark.parametrize("kw,want", [
    (dict(io=2), EDTYPE), (dict(rt=5), EDTYPE), (dict(M=-1), ESHAPE), (dict(D=-1), ESHAPE), (dict(eps=-1.0), ESHAPE),
    (dict(eps=math.nan), ESHAPE), (dict(eps=math.inf), ESHAPE), (dict(D=32769), EUNSUP), (dict(io=F32, rt=BF16), EUNSUP),
    (dict(residual=None), EUNSUP), (dict(M=1 << 26), ESHAPE), (dict(M=1 << 22, D=4097), ESHAPE), (dict(M=1 << 39, D=4), ESHAPE), (dict(x=None), ENULL),
    (dict(weight=None), ENULL), (dict(out=None), ENULL), (dict(x=ctypes.c_void_p((1 << 40) + 1)), EALIGN),
    (dict(residual=ctypes.c_void_p((2 << 40) + 2)), EALIGN), (dict(weight=ctypes.c_void_p((3 << 40) + 2)), EALIGN),
    (dict(out=X), EALIAS), (dict(residual_out=X), EALIAS), (dict(residual_out=W), EALIAS), (dict(out=R), EALIAS),
    (dict(residual_out=O), EALIAS), (dict(residual_out=ctypes.c_void_p((2 << 40) + 4)), EALIAS), (dict(M=0), OK)])
def test_norm_rejects(lib, call, kw, want):
    assert call(lib, **kw) == want


def test_norm_int8_rejects(lib):
    assert norm8(lib, scale=None) == ENULL
    assert norm8(lib, scale=X) == EALIAS and norm8(lib, scale=O) == EALIAS and norm8(lib, scale=RO) == EALIAS
    assert norm8(lib, scale=ctypes.c_void_p((6 << 40) + 2)) == EALIGN
    assert norm8(lib, D=0) == ESHAPE and norm8(lib, D=0, M=0) == OK
    assert norm(lib, D=0) == OK


@pytest.mark.parametrize("kw,want", [
    (dict(io=3), EDTYPE), (dict(ht=3), EDTYPE), (dict(M=-1), ESHAPE), (dict(eps=-1.0), ESHAPE), (dict(D=32769), EUNSUP),
    (dict(io=F32, ht=BF16), EUNSUP), (dict(ht=BF16), EUNSUP), (dict(dw=None), ENULL), (dict(dy=None), ENULL),
    (dict(h=None), ENULL), (dict(w=None), ENULL), (dict(dx=None), ENULL), (dict(ws=None), EWS), (dict(wsb=8), EWS),
    (dict(ws=ctypes.c_void_p((7 << 40) + 128)), EWS), (dict(dy=ctypes.c_void_p((1 << 40) + 1)), EALIGN),
    (dict(dx=X), EALIAS), (dict(dx=R), EALIAS), (dict(dr=DX), EALIAS), (dict(dw=W), EALIAS), (dict(ws=X), EALIAS),
    (dict(D=0), OK)])
def test_norm_bwd_rejects(lib, kw, want):
    a = dict(dy=X, h=R, w=W, dro=O, dx=DX, dr=DR, dw=S, ws=WS, wsb=1 << 30, M=4, D=64, eps=1e-5, io=BF16, ht=F32,
             stream=None)
    a.update(kw)
    assert lib.mamba_rms_norm_bwd(*a.values()) == want


def test_norm_bwd_workspace(lib):
    size = lib.mamba_rms_norm_bwd_workspace_size
    assert size(0, 64) == 0 and size(4, 0) == 0 and size(-1, 4) == 0 and size(4, 32769) == 0
    for M, D in [(1, 1), (3, 7), (100, 1024), (16384, 2560), (1 << 25, 768)]:
        assert 0 < size(M, D) <= 4096 * D * 4 and size(M, D) % (4 * D) == 0


@pytest.mark.parametrize("kw,want", [
    (dict(io=2), EDTYPE), (dict(B=-1), ESHAPE), (dict(cm=2), EUNSUP), (dict(K=32769), EUNSUP), (dict(L=1 << 25), ESHAPE), (dict(L=1 << 21, K=5000), ESHAPE), (dict(L=1 << 25, cm=1), ESHAPE),
    (dict(B=1 << 22, L=3, cm=1), ESHAPE),
    (dict(K=0), ESHAPE), (dict(B=0), OK), (dict(L=0, K=0), OK), (dict(x=None), ENULL), (dict(q=None), ENULL),
    (dict(s=None), ENULL), (dict(x=ctypes.c_void_p((1 << 40) + 1)), EALIGN), (dict(s=ctypes.c_void_p((6 << 40) + 1)), EALIGN),
    (dict(q=X), EALIAS), (dict(s=X), EALIAS), (dict(s=O), EALIAS)])
def test_quantize_rejects(lib, kw, want):
    a = dict(x=X, q=O, s=S, B=2, L=8, K=64, cm=0, io=BF16, stream=None)
    a.update(kw)
    assert lib.mamba_quantize_int8(*a.values()) == want


@pytest.mark.parametrize("kw,want", [
    (dict(ot=2), EDTYPE), (dict(M=-1), ESHAPE), (dict(K=-1), ESHAPE), (dict(batch=-1), ESHAPE), (dict(K=131072), EUNSUP),
    (dict(flags=4), EUNSUP), (dict(M=1 << 30, N=1 << 30), ESHAPE), (dict(M=1 << 20, N=1 << 20), ESHAPE), (dict(M=0), OK),
    (dict(N=0), OK), (dict(batch=0), OK), (dict(a=None), ENULL), (dict(b=None), ENULL), (dict(out=None), ENULL),
    (dict(sa=None), ENULL), (dict(sb=None), ENULL), (dict(sa=ctypes.c_void_p((3 << 40) + 2)), EALIGN),
    (dict(out=ctypes.c_void_p((5 << 40) + 1)), EALIGN), (dict(out=X), EALIAS), (dict(out=R), EALIAS), (dict(out=W), EALIAS),
    (dict(out=O), EALIAS)])
def test_matmul_rejects(lib, kw, want):
    a = dict(a=X, b=R, sa=W, sb=O, out=RO, batch=2, M=33, N=40, K=128, ot=BF16, flags=0, stream=None)
    a.update(kw)
    assert lib.mamba_int8_matmul(*a.values()) == want

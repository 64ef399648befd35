"""CPU checks of the microscaled 4-bit entry points: bad arguments are refused before
any HIP call."""
import ctypes

import pytest

import selective_state_space_80_amd as mamba

F32, BF16 = mamba.MAMBA_F32, mamba.MAMBA_BF16
OK, ENULL, ESHAPE, EDTYPE, EUNSUP, EALIGN, EALIAS, EWS, ELAUNCH, EDEV, ETIMEOUT = range(11)


@pytest.fixture(scope="module")
def lib():
    return mamba.load_library()


def _p(k, off=0):
    """Made-up device addresses, far apart: never dereferenced on the host."""
    return ctypes.c_void_p((k << 40) + off)


X, Q, S, A, B, SA, SB, O = (_p(k) for k in range(1, 9))


def quant(lib, **kw):
    a = dict(x=X, q=Q, s=S, B=2, L=100, K=300, cm=0, io=BF16, stream=None)
    a.update(kw)
    return lib.mamba_quantize_mxfp4(*a.values())


def dequant(lib, **kw):
    a = dict(q=Q, s=S, out=O, rows=100, K=300, io=BF16, stream=None)
    a.update(kw)
    return lib.mamba_dequantize_mxfp4(*a.values())


def matmul(lib, **kw):
    a = dict(a=A, b=B, sa=SA, sb=SB, out=O, batch=2, M=100, N=200, K=300, out_type=BF16, flags=0, stream=None)
    a.update(kw)
    return lib.mamba_mxfp4_matmul(*a.values())


@pytest.mark.parametrize("cm", [0, 1])
@pytest.mark.parametrize("kw,want", [
    (dict(io=2), EDTYPE), (dict(B=-1), ESHAPE), (dict(L=-1), ESHAPE), (dict(K=-1), ESHAPE), (dict(K=(1 << 23) + 1), EUNSUP),
    (dict(L=1 << 26, B=1, K=1 << 14), ESHAPE), (dict(L=1 << 39), ESHAPE), (dict(cm=2), EUNSUP), (dict(x=None), ENULL), (dict(q=None), ENULL), (dict(s=None), ENULL),
    (dict(x=_p(1, 1)), EALIGN), (dict(q=_p(2, 8)), EALIGN), (dict(s=_p(3, 4)), EALIGN), (dict(q=X), EALIAS), (dict(s=X), EALIAS),
    (dict(s=Q), EALIAS), (dict(s=_p(2, 200 * 256 - 8)), EALIAS), (dict(q=_p(1, 2 * 100 * 300 * 2 - 16)), EALIAS),
    (dict(B=0), OK), (dict(L=0), OK), (dict(K=0), OK)])
def test_quantise_rejects(lib, cm, kw, want):
    assert quant(lib, **{"cm": cm, **kw}) == want


@pytest.mark.parametrize("kw,want", [
    (dict(io=2), EDTYPE), (dict(rows=-1), ESHAPE), (dict(K=-1), ESHAPE), (dict(K=(1 << 23) + 1), EUNSUP), (dict(rows=1 << 28), ESHAPE),
    (dict(q=None), ENULL), (dict(s=None), ENULL), (dict(out=None), ENULL), (dict(q=_p(2, 8)), EALIGN), (dict(s=_p(3, 4)), EALIGN),
    (dict(out=_p(8, 1)), EALIGN), (dict(out=Q), EALIAS), (dict(out=S), EALIAS), (dict(rows=0), OK), (dict(K=0), OK)])
def test_dequantise_rejects(lib, kw, want):
    assert dequant(lib, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(out_type=2), EDTYPE), (dict(batch=-1), ESHAPE), (dict(M=-1), ESHAPE), (dict(N=-1), ESHAPE), (dict(K=-1), ESHAPE),
    (dict(K=(1 << 23) + 1), EUNSUP), (dict(flags=4), EUNSUP), (dict(batch=1, M=1 << 20, N=1 << 23), ESHAPE), (dict(a=None), ENULL),
    (dict(b=None), ENULL), (dict(sa=None), ENULL), (dict(sb=None), ENULL), (dict(out=None), ENULL), (dict(a=_p(4, 8)), EALIGN),
    (dict(b=_p(5, 4)), EALIGN), (dict(sa=_p(6, 4)), EALIGN), (dict(sb=_p(7, 1)), EALIGN), (dict(out=_p(8, 1)), EALIGN),
    (dict(out=A), EALIAS), (dict(out=B), EALIAS), (dict(out=SA), EALIAS), (dict(out=SB), EALIAS),
    (dict(out=_p(4, 2 * 100 * 256 - 2)), EALIAS), (dict(batch=0), OK), (dict(M=0), OK), (dict(N=0), OK)])
def test_product_rejects(lib, kw, want):
    assert matmul(lib, **kw) == want


def test_binding_refuses():
    """Metadata that does not fit, before the library is asked: on CPU tensors."""
    import torch
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    a, sa, b, sb = u8(5, 256), u8(2, 5, 8), u8(7, 256), u8(2, 7, 8)
    for bad in ((u8(5, 255), b, sa, sb), (u8(5, 128), b, u8(1, 5, 8), sb), (a.to(torch.int8), b, sa, sb), (a, b, u8(5, 2, 8), sb),
                (a, b, sa.float(), sb), (a.t(), b, sa, sb), (u8(2, 5, 256), u8(3, 7, 256), u8(2, 2, 5, 8), u8(2, 3, 7, 8)),
                (u8(256), b, u8(2, 8), sb), (a, b, sa, u8(2, 8, 7).transpose(1, 2))):
        with pytest.raises((ValueError, TypeError)):
            mamba.mxfp4_matmul(*bad)
    with pytest.raises(ValueError, match="GPU"):
        mamba.mxfp4_matmul(a, b, sa, sb)
    with pytest.raises(ValueError):
        mamba.dequantize_mxfp4(a, sa, 256)
    with pytest.raises(ValueError):
        mamba.dequantize_mxfp4(a, sa, 513)
    with pytest.raises(ValueError):
        mamba.quantize_mxfp4(torch.zeros(4, 5), channel_major=True)
    with pytest.raises(ValueError):
        mamba.quantize_mxfp4(torch.zeros(4, 5).t())
    with pytest.raises(ValueError):
        mamba.quantize_mxfp4(torch.zeros(4, 5), out=u8(4, 64))
    with pytest.raises(TypeError):
        mamba.quantize_mxfp4(torch.zeros(4, 5).half())

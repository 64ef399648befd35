"""CPU checks of the gated recurrence's entry points: bad arguments are refused before
any HIP call."""
import ctypes
import math

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


X, R, I, LAM, RB, IB, Z, H0, RESET, Y, HL, CK, DO, DHL, DX, DR, DI, DZ, DLAM, DRB, DIB, DH0, WS = (
    _p(k) for k in range(1, 24))


def fwd(lib, **kw):
    a = dict(x=X, r=R, i=I, lam=LAM, rb=RB, ib=IB, z=Z, h0=H0, reset=RESET, y=Y, hl=HL, ck=CK, ws=WS, nws=1 << 20, B=2, D=64, L=600, c=8.0,
             io=BF16, stream=None)
    a.update(kw)
    return lib.mamba_gated_scan_fwd(*a.values())


def bwd(lib, **kw):
    a = dict(x=X, r=R, i=I, lam=LAM, rb=RB, ib=IB, z=Z, h0=H0, reset=RESET, ck=CK, dout=DO, dhl=DHL, dx=DX, dr=DR, di=DI,
             dz=DZ, dlam=DLAM, drb=DRB, dib=DIB, dh0=DH0, ws=WS, nws=1 << 20, B=2, D=64, L=600, c=8.0, io=BF16, stream=None)
    a.update(kw)
    return lib.mamba_gated_scan_bwd(*a.values())


def step(lib, **kw):
    a = dict(h=H0, ho=HL, x=X, r=R, i=I, lam=LAM, rb=RB, ib=IB, z=Z, y=Y, B=2, D=64, c=8.0, io=BF16, stream=None)
    a.update(kw)
    return lib.mamba_gated_state_update(*a.values())


COMMON = [(dict(io=2), EDTYPE), (dict(B=-1), ESHAPE), (dict(D=-1), ESHAPE), (dict(c=-1.0), ESHAPE), (dict(c=math.nan), ESHAPE),
          (dict(c=math.inf), ESHAPE), (dict(x=None), ENULL), (dict(r=None), ENULL), (dict(i=None), ENULL), (dict(lam=None), ENULL),
          (dict(x=_p(1, 1)), EALIGN), (dict(r=_p(2, 1)), EALIGN), (dict(i=_p(3, 1)), EALIGN), (dict(lam=_p(4, 2)), EALIGN),
          (dict(rb=_p(5, 2)), EALIGN), (dict(ib=_p(6, 1)), EALIGN), (dict(z=_p(7, 1)), EALIGN), (dict(h0=_p(8, 2)), EALIGN)]


@pytest.mark.parametrize("kw,want", COMMON + [
    (dict(L=-1), ESHAPE), (dict(D=1 << 23), ESHAPE), (dict(L=1 << 39), ESHAPE), (dict(y=None), ENULL), (dict(y=_p(10, 1)), EALIGN),
    (dict(hl=_p(11, 2)), EALIGN), (dict(ck=_p(12, 2)), EALIGN), (dict(y=X), EALIAS), (dict(y=Z), EALIAS), (dict(y=RESET), EALIAS),
    (dict(hl=H0), EALIAS), (dict(hl=Y), EALIAS), (dict(ck=HL), EALIAS), (dict(ck=LAM), EALIAS), (dict(y=RB), EALIAS),
    (dict(y=_p(1, 2 * 64 * 600 * 2 - 2)), EALIAS), (dict(B=0), OK), (dict(D=0), OK), (dict(L=0, hl=None), OK),
    (dict(L=50000, ws=None), EWS), (dict(L=50000, nws=1024), EWS), (dict(L=50000, ws=_p(23, 128)), EWS),
    (dict(L=50000, ws=X), EALIAS), (dict(L=50000, ws=Y), EALIAS)])
def test_forward_rejects(lib, kw, want):
    assert fwd(lib, **kw) == want


@pytest.mark.parametrize("kw,want", COMMON[:-1] + [
    (dict(L=-1), ESHAPE), (dict(D=1 << 23), ESHAPE), (dict(dout=None), ENULL), (dict(dx=None), ENULL), (dict(dr=None), ENULL),
    (dict(di=None), ENULL), (dict(dz=None), ENULL), (dict(z=None), EUNSUP), (dict(dlam=None), ENULL), (dict(drb=None), ENULL),
    (dict(dib=None), ENULL), (dict(dh0=None), ENULL), (dict(dout=_p(13, 1)), EALIGN), (dict(dhl=_p(14, 1)), EALIGN),
    (dict(dx=_p(15, 1)), EALIGN), (dict(dh0=_p(22, 2)), EALIGN), (dict(ck=_p(12, 2)), EALIGN), (dict(ws=None), EWS),
    (dict(nws=255), EWS), (dict(ws=_p(23, 128)), EWS), (dict(ck=None, nws=2 * 64 * 3 * 4), EWS), (dict(dx=DO), EALIAS),
    (dict(dx=X), EALIAS), (dict(dr=DX), EALIAS), (dict(dz=DI), EALIAS), (dict(dlam=LAM), EALIAS), (dict(dh0=DHL), EALIAS),
    (dict(ws=X), EALIAS), (dict(ws=CK), EALIAS), (dict(dh0=H0), EALIAS), (dict(D=0), OK),
    (dict(B=0, D=1 << 24), ESHAPE)])
def test_backward_rejects(lib, kw, want):
    assert bwd(lib, **kw) == want


@pytest.mark.parametrize("kw,want", [(k, EALIGN if "h0" in k else w) for k, w in COMMON[:-1]] + [
    (dict(h=None), ENULL), (dict(ho=None), ENULL), (dict(y=None), ENULL), (dict(h=_p(8, 2)), EALIGN), (dict(ho=_p(11, 2)), EALIGN),
    (dict(y=X), EALIAS), (dict(y=H0), EALIAS), (dict(y=HL), EALIAS), (dict(ho=_p(8, 4)), EALIAS), (dict(ho=X), EALIAS),
    (dict(B=1 << 16, D=1 << 15), ESHAPE), (dict(B=0), OK), (dict(D=0), OK)])
def test_step_rejects(lib, kw, want):
    assert step(lib, **kw) == want


def test_sizes(lib):
    assert [lib.mamba_gated_scan_checkpoints(L) for L in (-1, 0, 1, 512, 513, 131072)] == [0, 0, 1, 1, 2, 256]
    size = lib.mamba_gated_scan_bwd_workspace_size
    assert size(2, 64, 600, 1) == 1536 and size(2, 64, 600, 0) == 1536 + 1024
    assert size(1, 64, 600, 1) == 0 and size(1, 64, 600, 0) == 512
    assert size(1, 64, 50000, 1) == 20 * 64 * 12 + 20 * 64 * 8  # 98 chunks in 20 parts of five
    assert lib.mamba_gated_scan_fwd_workspace_size(1, 64, 50000) == 20 * 64 * 8
    assert lib.mamba_gated_scan_fwd_workspace_size(3, 64, 50000) == 0 and lib.mamba_gated_scan_fwd_workspace_size(1, 64, 15872) == 0
    assert size(-1, 64, 600, 1) == 0 and size(1, 1 << 24, 1, 1) == 0


def test_binding_refuses():
    """Metadata that does not fit, before the library is asked: on CPU tensors."""
    import torch
    x, lam = torch.zeros(2, 3, 5), torch.zeros(3)
    call = mamba.gated_scan_fwd
    for bad in (dict(r=torch.zeros(2, 3, 4)), dict(r=torch.zeros(2, 3, 5).to(torch.bfloat16)), dict(lam=torch.zeros(4)),
                dict(lam=torch.zeros(3).double()), dict(z=torch.zeros(2, 5, 3).transpose(1, 2)), dict(h0=torch.zeros(3)),
                dict(reset=torch.zeros(2, 5)), dict(reset=torch.zeros(2, 3, dtype=torch.bool)), dict(r_bias=torch.zeros(2)),
                dict(out=torch.zeros(2, 3, 4)), dict(checkpoints=torch.zeros(2, 3, 2))):
        a = dict(x=x, r=x, i=x, lam=lam)
        a.update(bad)
        with pytest.raises((ValueError, TypeError)):
            call(**a)
    with pytest.raises(ValueError, match="GPU"):
        call(x, x, x, lam)
    with pytest.raises(ValueError):
        mamba.gated_scan_bwd(x, x, x, lam, torch.zeros(2, 3, 4))
    with pytest.raises(ValueError):
        mamba.gated_state_update(torch.zeros(2, 4), x[..., 0].contiguous(), x[..., 0].contiguous(), x[..., 0].contiguous(), lam)
    with pytest.raises((ValueError, TypeError)):
        mamba.gated_state_update(None, x[..., 0].contiguous(), x[..., 0].contiguous(), x[..., 0].contiguous(), lam)

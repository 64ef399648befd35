"""The gated recurrence where two to eight waves share a row, in every type and option; its
gradients at small and large lam; a padded sequence beside the same one without padding.
Against 64 bits with the bounds of gated_check.py."""
import pytest
import torch

import gated_check as C
from scan_check import say

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
GRADS = ("dx", "dr", "di", "dz", "dlam", "dr_bias", "di_bias", "dh0")
PER_CHANNEL = ("dlam", "dr_bias", "di_bias")


def _mamba():
    import selective_state_space_80_amd as mamba
    return mamba


def _call(p, which, *more, **kw):
    g = {k: None if v is None else v.cuda() for k, v in p.items()}
    return getattr(_mamba(), which)(g["x"], g["r"], g["i"], g["lam"], *more, r_bias=g["r_bias"], i_bias=g["i_bias"],
                                    z=g["z"], h0=g["h0"], reset=g["reset"], **kw)


def _forward(p, **kw):
    return _call(p, "gated_scan_fwd", return_last_state=True, return_checkpoints=True, **kw)


def _backward(p, q, **kw):
    return _call(p, "gated_scan_bwd", q["dout"].cuda(), dh_last=q["dh_last"].cuda(), **kw)


# more than 128 rows of 32 chunks or more: eight waves forward; backward four below 128 chunks, then eight
@pytest.mark.parametrize("io,gate,reset", [(BF16, False, 0.0), (BF16, True, 1e-3), (F32, True, 1e-3), (F32, False, 1e-3)])
@pytest.mark.parametrize("D,L", [(131, 16500), (130, 65700)])
def test_eight_waves(D, L, io, gate, reset):
    assert _mamba().gated_scan_fwd_workspace_size(1, D, L) == 0
    say(f"gated scan of eight waves {D} x {L} {io} gate={gate} reset={reset}")
    p = C.make(1, D, L, io, seed=D, gate=gate, reset=reset, decay=(0.99, 0.9999))
    q = C.gradient_inputs(p, 1)
    y, h_last, kept = _forward(p)
    got = _backward(p, q, checkpoints=kept)
    rows = [0, 64, D - 1]
    some = {k: (None if v is None else (v if k == "reset" else (v[:, rows].contiguous() if v.dim() > 1 else v[rows])))
            for k, v in p.items()}
    f, want = C.forward(some), C.backward(some, {k: v[:, rows].contiguous() for k, v in q.items()})
    parts = {"y": C.worst(y[:, rows], f["y"], f["y_err"]), "h_last": C.worst(h_last[:, rows], f["h_last"], f["h_last_err"])}
    for name in GRADS:
        if name in want:
            mine = got[name][rows] if name in PER_CHANNEL else got[name][:, rows]
            parts[name] = C.worst(mine, want[name], want[name + "_err"])
    say("  parts of the bounds: " + ", ".join(f"{k} {v:.2f}" for k, v in parts.items()))
    assert max(parts.values()) <= 1.0, parts


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("D,L", [(4, 3600), (4, 8200), (130, 16500), (130, 65700)])
def test_waves_keep_sequences_apart(D, L, io):
    """NaN and infinities of one packed sequence, where two, four and eight waves share a row."""
    assert _mamba().gated_scan_fwd_workspace_size(1, D, L) == 0
    p = C.make(1, D, L, io, seed=L)
    q = C.gradient_inputs(p, 2)
    lo, hi = L // 3, 2 * L // 3
    p["reset"] = torch.zeros(1, L, dtype=torch.bool)
    p["reset"][0, [0, lo, hi]] = True
    p["h0"][:] = torch.nan
    clean = {k: (v.clone() if v is not None else None) for k, v in p.items()}
    p["x"][0, 0, lo + 1] = torch.nan
    p["x"][0, 1, lo + 700] = torch.inf
    p["r"][0, 2, hi - 600] = torch.nan
    p["x"][0, 3, hi - 1] = -torch.inf
    y, h_last, kept = _forward(p)
    got = _backward(p, q, checkpoints=kept)
    y0, last0, kept0 = _forward(clean)
    got0 = _backward(clean, q, checkpoints=kept0)
    outside = torch.ones(L, dtype=torch.bool)
    outside[lo:hi] = False
    assert torch.isfinite(y0).all() and torch.isnan(y[0, 0, lo + 1:hi]).all()
    assert torch.equal(y[..., outside], y0[..., outside]) and torch.equal(h_last, last0)
    for name in ("dx", "dr", "di", "dz"):
        assert torch.isfinite(got0[name]).all()
        assert torch.equal(got[name][..., outside], got0[name][..., outside]), name


@pytest.mark.parametrize("lam,c", [(-84.0, 8.0), (-81.0, 0.25)] + [(lam, c) for lam in (-79.0, -30.0, 0.0, 30.0, 90.0)
                                                                   for c in (0.25, 8.0)])
def test_gradient_at_lam(lam, c):
    """Below -80 the slope sigmoid(lam) / softplus(lam) is taken as 1; v stays in fp32's normal
    range (8 e^-84 sigmoid(-4) = 5e-38, e^-81 sigmoid(-4) / 4 = 3e-38)."""
    p = C.make(2, 3, 70, F32, seed=8)
    p["lam"] = torch.full((3,), lam)
    say(f"gated scan gradient at lam={lam} c={c}")
    q = C.gradient_inputs(p, 9)
    want, got = C.backward(p, q, c), _backward(p, q, c=c)
    parts = {name: C.worst(got[name], want[name], want[name + "_err"]) for name in GRADS}
    say("  parts of the bounds: " + ", ".join(f"{k} {v:.2f}" for k, v in parts.items()))
    assert max(parts.values()) <= 1.0, parts
    assert lam > 0 or got["dlam"].abs().min() > 0


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("length", [1, 8, 137, 299])
def test_padded_sequence_is_the_short_one(io, length):
    """Both calls are within their bounds of the same 64 bits; and the state is what the short one ends in."""
    p = C.make(2, 6, 300, io, seed=11)
    p["r"][1, :, length:] = -torch.inf
    y, h_last, _ = _forward(p)
    short = {k: (v[1:2, :, :length].contiguous() if v is not None and v.dim() == 3 else v) for k, v in p.items()}
    short["h0"] = p["h0"][1:2].contiguous()
    y1, last1, _ = _forward(short)
    f = C.forward(short)
    for got, want, err in ((y1, f["y"], f["y_err"]), (y[1:2, :, :length], f["y"], f["y_err"]),
                           (last1, f["h_last"], f["h_last_err"]), (h_last[1:2], f["h_last"], f["h_last_err"])):
        assert C.worst(got, want, err) <= 1

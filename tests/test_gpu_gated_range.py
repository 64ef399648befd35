"""The gated recurrence at the ends of its parameters' range, against 64 bits with the
bounds of gated_check.py.  Those know no underflow of v, whose root m = sqrt(2 v) is: below
lam = -104 softplus(lam) < 2^-149 is 0 in fp32, and m with it, where 64 bits still have m =
7e-24.  There, and where a parameter is infinite, the 64-bit side takes a finite value whose
gates are the same in fp32 and far past it: softplus(-700) = 1e-304, m below 1e-151, and a decay of
1e38 leaves nothing of a state, as one of infinity does."""
import pytest
import torch

import gated_check as C
from scan_check import say

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
INF = float("inf")
GRADS = ("dx", "dr", "di", "dz", "dlam", "dr_bias", "di_bias", "dh0")
PARAMETERS = ("lam", "r_bias", "i_bias")


def _mamba():
    import selective_state_space_80_amd as mamba
    return mamba


def _call(p, which, *more, **kw):
    g = {k: None if v is None else v.cuda() for k, v in p.items()}
    return getattr(_mamba(), which)(g["x"], g["r"], g["i"], g["lam"], *more, r_bias=g["r_bias"], i_bias=g["i_bias"],
                                    z=g["z"], h0=g["h0"], reset=g["reset"], **kw)


def _step(p, c):
    """The first step of p by the single-step call: (y, state)."""
    g = {k: (v[..., 0].contiguous() if v is not None and v.dim() == 3 else v) for k, v in p.items()}
    g = {k: None if v is None else v.cuda() for k, v in g.items()}
    h = torch.empty_like(g["h0"])
    y = _mamba().gated_state_update(g["h0"], g["x"], g["r"], g["i"], g["lam"], r_bias=g["r_bias"], i_bias=g["i_bias"],
                                    z=g["z"], c=c, h_out=h)
    return y, h


def _far(p):
    """p with finite parameters that mean the same."""
    out = dict(p, lam=torch.where(p["lam"] < -104.0, -700.0, p["lam"].clamp(max=3e38)))
    for name in ("r_bias", "i_bias"):
        if p[name] is not None:
            out[name] = p[name].clamp(-700.0, 700.0)
    return out


def _check(p, seed, c=8.0, forgets=()):
    """Forward, gradient and single step; forgets: channels whose every step has v above 1e4, so
    that a is 0 (to any number of bits that fp32 has) and dr and dlam are 0."""
    far = _far(p)
    f, q = C.forward(far, c), C.gradient_inputs(p, seed)
    want = C.backward(far, q, c)
    y, h_last, kept = _call(p, "gated_scan_fwd", c=c, return_last_state=True, return_checkpoints=True)
    parts = {"y": C.worst(y, f["y"], f["y_err"]), "h_last": C.worst(h_last, f["h_last"], f["h_last_err"])}
    forgets = torch.tensor(sorted(forgets), dtype=torch.long)
    for kw in (dict(checkpoints=kept), {}):
        got = _call(p, "gated_scan_bwd", q["dout"].cuda(), dh_last=q["dh_last"].cuda(), c=c, **kw)
        for name in GRADS:
            if name not in want:
                assert got[name] is None
                continue
            part = C.worst(got[name], want[name], want[name + "_err"])
            parts[name] = max(part, parts.get(name, 0.0))
        assert not got["dr"][:, forgets].any() and not got["dlam"][forgets].any()
    first = {k: (v[..., :1].contiguous() if v is not None and v.dim() == 3 else v) for k, v in p.items()}
    first["reset"] = None
    f1 = C.forward(_far(first), c)
    y1, h1 = _step(first, c)
    parts["step"] = max(C.worst(y1, f1["y"][..., 0], f1["y_err"][..., 0]), C.worst(h1, f1["h_last"], f1["h_last_err"]))
    say("  parts of the bounds: " + ", ".join(f"{k} {v:.2f}" for k, v in parts.items()))
    assert max(parts.values()) <= 1.0, parts


# lengths that fill the lanes of every kind of row: groups of 4, 16, 32 and 64 lanes, two and
# four waves a row, and parts of a row (from 15873 steps on)
WHOLE = [32, 128, 256, 1024, 4096, 8192, 16384]
# not between 709 and 1e4, where the 64-bit side's e^lam is infinite
LARGE = [s * v for v in (1.5e2, 2.5e2, 6e2, 2e4, 3e9, 1e10, 3.3e10, 1e12, 1e20, 1e30, 1e37) for s in (1, -1)] + [-3e38, -INF]


@pytest.mark.parametrize("io,reset", [(F32, 0.0), (BF16, 0.01)])
@pytest.mark.parametrize("L", WHOLE)
def test_large_lam(L, io, reset):
    """lam of any size: a channel that keeps its state, or one that forgets it."""
    say(f"gated scan large lam L={L} {io}")
    p = C.make(1, len(LARGE), L, io, seed=L, gate=io == BF16, reset=reset)
    p["lam"] = torch.tensor(LARGE)
    _check(p, L + 1, forgets=[k for k, v in enumerate(LARGE) if v > 1e8])


@pytest.mark.parametrize("size", [1e9, 1e10, 1e20, 1e30])
def test_large_lam_and_small_c(size):
    """c softplus(lam) between 0.1 and 4: ordinary decays."""
    say(f"gated scan lam {size}, c {1 / size}")
    p = C.make(2, 24, 1024, F32, seed=3)
    p["lam"] = torch.linspace(0.1, 4.0, 24) * size
    _check(p, 4, c=float(torch.tensor(1 / size)))


def test_nan_lam_stays_in_its_channel():
    p = C.make(2, 4, 512, F32, seed=5)
    clean = _call(p, "gated_scan_fwd")
    lam = p["lam"].clone()
    lam[1] = torch.nan
    y = _call(dict(p, lam=lam), "gated_scan_fwd")
    others = torch.tensor([0, 2, 3])
    assert torch.isnan(y[:, 1]).all() and torch.equal(y[:, others], clean[:, others])
    y1, h1 = _step(dict(p, lam=lam), 8.0)
    assert torch.isnan(y1[:, 1]).all() and torch.isnan(h1[:, 1]).all() and torch.isfinite(h1[:, others]).all()


# (lam, r_bias, i_bias): gates that are always open or shut, rates past the largest float
ENDS = [(-3.0, INF, 0.5), (-3.0, -INF, 0.5), (-3.0, 3e38, 0.5), (-3.0, -3e38, 0.5), (INF, 0.3, -0.2), (3e38, 0.3, -0.2),
        (INF, INF, 0.1), (INF, -INF, 0.1), (-INF, INF, 0.1), (-3.0, 0.2, INF), (-3.0, 0.2, -INF), (INF, INF, INF), (-2.0, 0.1, 0.4)]
FORGETS = [4, 5, 6, 11]  # channels of those
# one step, and lengths that leave a part of a lane, of its group, of a chunk, of the waves of a row and of a row's last part
ODD = [1, 5, 30, 32, 100, 200, 257, 300, 511, 700, 1024, 3600, 8200, 16400]


@pytest.mark.parametrize("io,reset", [(F32, 0.0), (BF16, 0.02)])
@pytest.mark.parametrize("L", ODD)
def test_infinite_parameters(L, io, reset):
    """Infinite parameters give the same at every length, and r = -inf leaves the state beside them too."""
    say(f"gated scan infinite parameters L={L} {io}")
    p = C.make(2, len(ENDS), L, io, seed=L, gate=io == BF16, reset=reset)
    for k, name in enumerate(PARAMETERS):
        p[name] = torch.tensor([e[k] for e in ENDS])
    p["r"][1, :, 2 * L // 3:] = -INF
    _check(p, L + 1, forgets=FORGETS)


@pytest.mark.parametrize("c,lam", [(3e38, 5.0), (1e30, 1e20), (1e-30, INF)])
def test_rates_past_the_largest_float(c, lam):
    say(f"gated scan c={c} lam={lam}")
    p = C.make(1, 3, 700, F32, seed=9, reset=0.01)
    p["lam"] = torch.tensor([lam, lam, -INF])
    _check(p, 10, c=c, forgets=[0, 1])


@pytest.mark.parametrize("name", PARAMETERS)
def test_nan_parameters_stay_in_their_channel(name):
    for L in (20, 700):
        p = C.make(2, 4, L, F32, seed=12, reset=0.02)
        q = C.gradient_inputs(p, 13)
        clean, clean_last = _call(p, "gated_scan_fwd", return_last_state=True)
        bad = dict(p, **{name: p[name].clone()})
        bad[name][2] = torch.nan
        y, last = _call(bad, "gated_scan_fwd", return_last_state=True)
        others = torch.tensor([0, 1, 3])
        assert torch.isnan(y[:, 2]).all() or name != "i_bias" and torch.isnan(y[:, 2]).any()
        assert torch.equal(y[:, others], clean[:, others]) and torch.equal(last[:, others], clean_last[:, others])
        a, b = (_call(t, "gated_scan_bwd", q["dout"].cuda()) for t in (p, bad))
        for g in GRADS:
            across = (lambda t: t[others]) if g in ("dlam", "dr_bias", "di_bias") else (lambda t: t[:, others])
            assert torch.equal(across(a[g]), across(b[g])), g


@pytest.mark.parametrize("L", [40, 700, 3600, 16400])
def test_nan_meets_a_channel_that_forgets(L):
    """0 times NaN: a decay to nothing is no reset, and drops no NaN; a reset behind it does."""
    p = C.make(1, 2, L, F32, seed=14)
    p["lam"] = torch.tensor([INF, 3e38])
    p["reset"] = torch.zeros(1, L, dtype=torch.bool)
    p["reset"][0, L // 2] = True
    p["x"][0, :, 3] = torch.nan
    y, last = _call(p, "gated_scan_fwd", return_last_state=True)
    assert torch.isnan(y[..., 3:L // 2]).all() and torch.isfinite(y[..., :3]).all()
    assert torch.isfinite(y[..., L // 2:]).all() and torch.isfinite(last).all()


@pytest.mark.parametrize("L", [20, 300, 700, 3600, 16400])
def test_an_infinite_state(L):
    """It is infinite, then from where a decay over several steps leaves fp32's range NaN, and
    never finite again without a reset; what is before it and beside it stays as it is."""
    p = C.make(1, 3, L, F32, seed=15, gate=False, reset=1e-9)  # no reset: the variant that has them
    assert not p["reset"].any()
    clean, clean_last = _call(p, "gated_scan_fwd", return_last_state=True)
    at = L // 3
    bad = dict(p, x=p["x"].clone(), h0=p["h0"].clone())
    bad["x"][0, 1, at] = INF
    bad["h0"][0, 2] = -INF
    for reset in (p["reset"], None):
        y, last = _call(dict(bad, reset=reset), "gated_scan_fwd", return_last_state=True)
        assert torch.equal(y[0, 0], clean[0, 0]) and torch.equal(y[0, 1, :at], clean[0, 1, :at])
        assert y[0, 1, at] == INF and y[0, 2, 0] == -INF
        for t in (y[0, 1, at:], y[0, 2], last[0, 1:]):
            assert not torch.isfinite(t).any()
        assert not (y[0, 1] == -INF).any() and not (y[0, 2] == INF).any()


def test_an_infinite_state_step_by_step():
    """As long as a step's own decay is in fp32's range, it stays infinite."""
    p = C.make(1, 3, 400, F32, seed=16, gate=False, biases=False)
    g = {k: None if v is None else v.cuda() for k, v in p.items()}
    h = torch.tensor([[INF, -INF, 1.0]], device="cuda")
    for t in range(400):
        y = _mamba().gated_state_update(h, *(g[n][..., t].contiguous() for n in ("x", "r", "i")), g["lam"])
        assert torch.equal(y, h)
    assert h[0, 0] == INF and h[0, 1] == -INF and torch.isfinite(h[0, 2])

"""GPU checks of the gated linear recurrence (forward, backward, single step) against
64 bits step by step; the bounds are derived in gated_check.py."""
import pytest
import torch

import gated_check as C
from scan_check import say

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
GRADS = ("dx", "dr", "di", "dz", "dlam", "dr_bias", "di_bias", "dh0")


def _cuda(p):
    return {k: None if v is None else v.cuda() for k, v in p.items()}


def _mamba():
    import selective_state_space_80_amd as mamba
    return mamba


def _forward(p, **kw):
    g = _cuda(p)
    return _mamba().gated_scan_fwd(g["x"], g["r"], g["i"], g["lam"], r_bias=g["r_bias"], i_bias=g["i_bias"], z=g["z"],
                                   h0=g["h0"], reset=g["reset"], **kw)


def _backward(p, q, **kw):
    g, d = _cuda(p), _cuda(q)
    return _mamba().gated_scan_bwd(g["x"], g["r"], g["i"], g["lam"], d["dout"], r_bias=g["r_bias"], i_bias=g["i_bias"],
                                   z=g["z"], h0=g["h0"], reset=g["reset"], dh_last=d["dh_last"], **kw)


def _check_both(p, seed, last=True, c=8.0):
    y, h_last, kept = _forward(p, return_last_state=True, return_checkpoints=True, c=c)
    f = C.forward(p, c)
    parts = {"y": C.worst(y, f["y"], f["y_err"]), "h_last": C.worst(h_last, f["h_last"], f["h_last_err"])}
    q = C.gradient_inputs(p, seed, last)
    want = C.backward(p, q, c)
    got = _backward(p, q, checkpoints=kept, c=c)
    for name in GRADS:
        if name in want:
            parts[name] = C.worst(got[name], want[name], want[name + "_err"])
        else:
            assert got[name] is None
    say("  parts of the bounds: " + ", ".join(f"{k} {v:.2f}" for k, v in parts.items()))
    assert max(parts.values()) <= 1.0, parts


# lengths: one token, inside a lane, the groups of 4, 16, 32 and 64 lanes and their ends, chunks and their ends
LENGTHS = [1, 2, 7, 8, 9, 31, 32, 33, 127, 128, 129, 255, 256, 257, 511, 512, 513, 1000, 1024, 1537, 2048, 2049]


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("L", LENGTHS)
def test_lengths(L, io):
    say(f"gated scan L={L} {io}")
    _check_both(C.make(2, 5, L, io, seed=L, reset=0.02 if L % 2 else 0.0), seed=L + 1)


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("reset", [0.0, 0.01, 1.0])
@pytest.mark.parametrize("h0,biases,last", [(False, False, False), (True, True, True)])
def test_options(io, gate, reset, h0, biases, last):
    say(f"gated scan options {io} gate={gate} reset={reset} h0={h0}")
    for B, D, L in [(3, 7, 40), (1, 3, 700), (2, 2, 2100)]:
        _check_both(C.make(B, D, L, io, seed=5, gate=gate, h0=h0, biases=biases, reset=reset), seed=6, last=last)


@pytest.mark.parametrize("B,D,L", [(1, 1, 600), (2, 2050, 520), (1, 4100, 130), (5, 1030, 17), (2, 2049, 1025)])
def test_rows(B, D, L):
    """Rows that leave a workgroup part empty, and enough of them for one wave a row."""
    say(f"gated scan rows {B} x {D} x {L}")
    _check_both(C.make(B, D, L, F32, seed=D, reset=0.01), seed=1)


@pytest.mark.parametrize("decay", [(1 - 1e-7, 1 - 1e-6), (1 - 1e-4, 1 - 1e-3), (1e-12, 1e-3), (1e-40, 1e-30)])
@pytest.mark.parametrize("spread", [0.0, 3.0])
def test_decays(decay, spread):
    """Memories of millions of steps and of none; gates that never change, or far apart."""
    say(f"gated scan decays {decay} spread {spread}")
    _check_both(C.make(1, 4, 3000, F32, seed=3, gate=False, decay=decay, spread=spread), seed=4)


@pytest.mark.parametrize("lam", [-90.0, -30.0, 0.0, 30.0, 90.0])
@pytest.mark.parametrize("c", [0.0, 0.25, 8.0])
def test_lam(lam, c):
    p = C.make(2, 3, 70, F32, seed=8)
    p["lam"] = torch.full((3,), lam)
    say(f"gated scan lam={lam} c={c}")
    f = C.forward(p, c)
    y, h_last = _forward(p, return_last_state=True, c=c)
    assert C.worst(y, f["y"], f["y_err"]) <= 1 and C.worst(h_last, f["h_last"], f["h_last_err"]) <= 1
    got = _backward(p, C.gradient_inputs(p, 9), c=c)
    assert all(torch.isfinite(got[n]).all() for n in GRADS)


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("padding", [None, 3e38])
def test_padded_tokens_leave_the_state(io, padding):
    """r = -inf: the state, its gradient and everything behind are as without the token,
    whatever finite input it has."""
    p = C.make(2, 6, 300, io, seed=11)
    q = C.gradient_inputs(p, 12)
    lengths = (300, 137)
    for b, n in enumerate(lengths):
        p["r"][b, :, n:] = -torch.inf
        if padding:
            p["x"][b, :, n:] = padding
    y, h_last, kept = _forward(p, return_last_state=True, return_checkpoints=True)
    got = _backward(p, q, checkpoints=kept)
    n = lengths[1]
    assert torch.equal(got["dr"][1, :, n:].cpu(), torch.zeros(6, 300 - n, dtype=io))
    short = {k: (v[1:2, :, :n].contiguous() if v is not None and v.dim() == 3 else v) for k, v in p.items()}
    short["h0"] = p["h0"][1:2]
    y1, last1 = _forward(short, return_last_state=True)
    f = C.forward(short)
    assert C.worst(y[1:2, :, :n], f["y"], f["y_err"]) <= 1
    assert C.worst(h_last[1:2], f["h_last"], f["h_last_err"]) <= 1
    want = C.backward(p, q)
    for name in GRADS:
        assert C.worst(got[name], want[name], want[name + "_err"]) <= 1, name


@pytest.mark.parametrize("L", [24, 100, 200, 1700])
def test_reset_keeps_sequences_apart(L):
    """NaN and infinities of one packed sequence reach neither its neighbours' outputs nor gradients."""
    p = C.make(1, 4, L, F32, seed=13, reset=0.0)
    q = C.gradient_inputs(p, 14)
    lo, hi = L // 3, 2 * L // 3
    p["reset"] = torch.zeros(1, L, dtype=torch.bool)
    p["reset"][0, [0, lo, hi]] = True
    p["h0"][:] = torch.nan
    clean = {k: (v.clone() if v is not None else None) for k, v in p.items()}
    p["x"][0, 0, lo + 1] = torch.nan
    p["x"][0, 1, lo + 1] = torch.inf
    p["r"][0, 2, lo + 2] = torch.nan
    p["x"][0, 3, hi - 1] = -torch.inf
    y, h_last, kept = _forward(p, return_last_state=True, return_checkpoints=True)
    got = _backward(p, q, checkpoints=kept)
    y0, last0, kept0 = _forward(clean, return_last_state=True, return_checkpoints=True)
    got0 = _backward(clean, q, checkpoints=kept0)
    outside = torch.ones(L, dtype=torch.bool)
    outside[lo:hi] = False
    assert torch.isfinite(y0).all() and torch.isnan(y[0, 0, lo + 1:hi]).all()
    assert torch.equal(y[..., outside], y0[..., outside]) and torch.equal(h_last, last0)
    for name in ("dx", "dr", "di", "dz"):
        assert torch.equal(got[name][..., outside], got0[name][..., outside]), name
    assert torch.equal(got["dh0"], torch.zeros_like(got["dh0"]))


def test_checkpoints_are_the_states():
    p = C.make(2, 3, 1500, F32, seed=15, reset=0.005)
    _, kept = _forward(p, return_checkpoints=True)
    f = C.forward(p)
    assert kept.shape == (2, 3, 3)
    assert torch.equal(kept[..., 0].cpu(), p["h0"])
    for k, t in ((1, 511), (2, 1023)):
        assert C.worst(kept[..., k], f["h"][..., t], f["h_err"][..., t] + 1e-37) <= 1


@pytest.mark.parametrize("B,D,L", [(2, 3, 20), (1, 5, 1300)])
def test_gradient_without_checkpoints_is_the_same(B, D, L):
    p = C.make(B, D, L, BF16, seed=16, reset=0.01)
    q = C.gradient_inputs(p, 17)
    _, kept = _forward(p, return_checkpoints=True)
    a, b = _backward(p, q, checkpoints=kept), _backward(p, q)
    assert all(torch.equal(a[n], b[n]) for n in GRADS)


def test_gradient_against_differences():
    """Central differences of the library's own forward pass in fp32 along random directions:
    step e leaves the third derivative, e^2 = 1e-4 of the second's size with the cancellation of
    the sum, and the outputs' rounding 1e-6 / e: below 1 %."""
    p = C.make(2, 6, 160, F32, seed=18, spread=1.0)
    q = C.gradient_inputs(p, 19)
    got = _backward(p, q)

    def loss(p):
        y, last = _forward(p, return_last_state=True)
        return (y.double().cpu() * q["dout"].double()).sum() + (last.double().cpu() * q["dh_last"].double()).sum()

    gen = torch.Generator().manual_seed(20)
    for name, grad in (("x", "dx"), ("r", "dr"), ("i", "di"), ("z", "dz"), ("lam", "dlam"), ("r_bias", "dr_bias"),
                       ("i_bias", "di_bias"), ("h0", "dh0")):
        # along the gradient itself and a random direction: no cancellation hides it
        e = 1e-2
        v = got[grad].cpu() / got[grad].cpu().norm() + 0.1 * torch.nn.functional.normalize(
            torch.randn(p[name].shape, generator=gen).flatten(), dim=0).view(p[name].shape)
        up, down = ({**p, name: p[name] + s * e * v} for s in (1, -1))
        change = (loss(up) - loss(down)) / (2 * e)
        along = (got[grad].double().cpu() * v.double()).sum()
        say(f"  {name}: {along.item():.5f} against {change.item():.5f}")
        assert abs(along - change) <= 1e-2 * abs(change), name


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("gate", [False, True])
@pytest.mark.parametrize("B,D", [(1, 1), (1, 2560), (3, 771), (256, 130), (33, 4096), (257, 5120)])
def test_step(io, gate, B, D):
    say(f"gated step {B} x {D} {io} gate={gate}")
    p = C.make(B, D, 1, io, seed=D, gate=gate)
    f = C.forward(p)
    g = {k: (v[..., 0].contiguous() if v is not None and v.dim() == 3 else v) for k, v in _cuda(p).items()}
    args = (g["x"], g["r"], g["i"], g["lam"])
    kw = dict(r_bias=g["r_bias"], i_bias=g["i_bias"], z=g["z"])
    h = g["h0"].clone()
    fresh = torch.full_like(h, torch.nan)
    y = _mamba().gated_state_update(h, *args, h_out=fresh, **kw)
    assert torch.equal(h, g["h0"])
    assert C.worst(y, f["y"][..., 0], f["y_err"][..., 0]) <= 1
    assert C.worst(fresh, f["h_last"], f["h_last_err"]) <= 1
    y2 = _mamba().gated_state_update(h, *args, **kw)
    assert torch.equal(h, fresh) and torch.equal(y, y2)


def test_steps_are_the_scan():
    """A scan of 40 steps, and 40 single steps: both within the bounds."""
    p = C.make(3, 70, 40, F32, seed=21)
    f = C.forward(p)
    g = _cuda(p)
    h = g["h0"].clone()
    ys = [_mamba().gated_state_update(h, *(g[n][..., t].contiguous() for n in ("x", "r", "i")), g["lam"],
                                      r_bias=g["r_bias"], i_bias=g["i_bias"], z=g["z"][..., t].contiguous())
          for t in range(40)]
    assert C.worst(torch.stack(ys, -1), f["y"], f["y_err"]) <= 1
    assert C.worst(h, f["h_last"], f["h_last_err"]) <= 1


def test_empty():
    mamba = _mamba()
    p = C.make(2, 3, 0, F32, seed=1, gate=False)
    y, h_last, kept = _forward(p, return_last_state=True, return_checkpoints=True)
    assert y.shape == (2, 3, 0) and kept.shape == (2, 3, 0) and torch.equal(h_last.cpu(), p["h0"])
    q = C.gradient_inputs(p, 2)
    got = _backward(p, q)
    assert torch.equal(got["dh0"].cpu(), q["dh_last"])
    assert all(torch.equal(got[n].cpu(), torch.zeros(3)) for n in ("dlam", "dr_bias", "di_bias"))
    none = torch.empty(0, 3, 5, device="cuda")
    lam = torch.zeros(3, device="cuda")
    got = mamba.gated_scan_bwd(none, none, none, lam, none)
    assert torch.equal(got["dlam"].cpu(), torch.zeros(3))
    assert mamba.gated_scan_fwd(none, none, none, lam).shape == (0, 3, 5)


def test_offsets_past_32_bits():
    """A row longer than 2^32 bytes into the tensor: the last row of 3 x 1 x 2^30 in bf16."""
    mamba = _mamba()
    L = 1 << 30
    x = torch.zeros(3, 1, L, dtype=BF16, device="cuda")
    x[2, 0, -700:] = 1.0
    lam = torch.full((1,), -2.0, device="cuda")
    y, last = mamba.gated_scan_fwd(x, x, x, lam, return_last_state=True)
    tail = x[2:, :, -700:].contiguous()
    want, want_last = mamba.gated_scan_fwd(tail, tail, tail, lam, return_last_state=True)
    assert not y[:2].any() and not y[2, 0, :-700].any()
    assert (y[2, 0, -700:].float() - want[0, 0].float()).abs().max() <= 2.0 ** -7 * want.float().abs().max()
    assert abs(last[2, 0] - want_last[0, 0]) <= 1e-5 * abs(want_last[0, 0])


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("L", [3600, 8200, 15872])
def test_waves_that_share_a_row(io, L):
    """Two and four waves a row, the last round of chunks not full."""
    say(f"gated scan L={L} {io}")
    _check_both(C.make(1, 3, L, io, seed=L, gate=io == BF16, reset=1e-3 if L % 16 else 0.0), seed=L + 1)


@pytest.mark.parametrize("io", [F32, BF16])
@pytest.mark.parametrize("B,D,L,reset", [(1, 3, 15873, 0.0), (2, 2, 16400, 1e-3), (1, 5, 40000, 1e-4), (1, 1, 70001, 0.0)])
def test_rows_in_parts(io, B, D, L, reset):
    """Few rows of many steps: parts of a row on different workgroups, joined by their maps."""
    assert _mamba().gated_scan_fwd_workspace_size(B, D, L) > 0
    say(f"gated scan in parts {B} x {D} x {L} {io}")
    p = C.make(B, D, L, io, seed=L, gate=io == F32, reset=reset, decay=(0.99, 0.99999))
    _check_both(p, seed=L + 1)
    q = C.gradient_inputs(p, 3)
    a = _backward(p, q, checkpoints=_forward(p, return_checkpoints=True)[1])
    b = _backward(p, q)
    assert all(torch.equal(a[n], b[n]) for n in GRADS if a[n] is not None)


def test_parts_keep_sequences_apart():
    """NaN of one packed sequence, in the parts' maps and in the state that enters the row."""
    L, lo, hi = 30000, 9001, 20003
    p = C.make(1, 2, L, F32, seed=50)
    q = C.gradient_inputs(p, 51)
    p["reset"] = torch.zeros(1, L, dtype=torch.bool)
    p["reset"][0, [0, lo, hi]] = True
    p["h0"][:] = torch.nan
    clean = {k: (v.clone() if v is not None else None) for k, v in p.items()}
    p["x"][0, 0, lo + 5] = torch.nan
    p["r"][0, 1, hi - 7000] = torch.nan
    y, h_last, kept = _forward(p, return_last_state=True, return_checkpoints=True)
    got = _backward(p, q, checkpoints=kept)
    y0, last0, kept0 = _forward(clean, return_last_state=True, return_checkpoints=True)
    got0 = _backward(clean, q, checkpoints=kept0)
    outside = torch.ones(L, dtype=torch.bool)
    outside[lo:hi] = False
    assert torch.isfinite(y0).all() and torch.isnan(y[0, 0, lo + 5:hi]).all()
    assert torch.equal(y[..., outside], y0[..., outside]) and torch.equal(h_last, last0)
    for name in ("dx", "dr", "di", "dz"):
        assert torch.equal(got[name][..., outside], got0[name][..., outside]), name


@pytest.mark.parametrize("D,L", [(600, 20000), (200, 33000), (130, 9000), (130, 66000)])
def test_many_rows_of_many_chunks(D, L):
    """Four and eight waves a row, forward and backward, rows in more than one workgroup a CU."""
    assert _mamba().gated_scan_fwd_workspace_size(1, D, L) == 0
    p = C.make(1, D, L, F32, seed=40, gate=False)
    q = C.gradient_inputs(p, 41)
    y, kept = _forward(p, return_checkpoints=True)
    got = _backward(p, q, checkpoints=kept)
    rows = [0, 1, 63, 64, 99, D - 1]
    some = {k: (None if v is None else (v[:, rows].contiguous() if v.dim() > 1 else v[rows])) for k, v in p.items()}
    sq = {k: v[:, rows].contiguous() for k, v in q.items()}
    f, want = C.forward(some), C.backward(some, sq)
    assert C.worst(y[:, rows], f["y"], f["y_err"]) <= 1
    for name in ("dx", "dr", "di", "dh0"):
        assert C.worst(got[name][:, rows], want[name], want[name + "_err"]) <= 1, name
    for name in ("dlam", "dr_bias", "di_bias"):
        assert C.worst(got[name][rows], want[name], want[name + "_err"]) <= 1, name


@pytest.mark.parametrize("B,D,L", [(2, 5, 90), (1, 3, 20000)])
def test_the_callers_own_buffers(B, D, L):
    """Outputs, workspaces and resets (any non-zero byte) that the caller brings."""
    mamba = _mamba()
    p = C.make(B, D, L, BF16, seed=60, reset=0.01)
    q = C.gradient_inputs(p, 61)
    y, last, kept = _forward(p, return_last_state=True, return_checkpoints=True)
    got = _backward(p, q, checkpoints=kept)
    marks = (p["reset"].to(torch.uint8) * torch.arange(1, L + 1) % 256).to(torch.uint8)
    own = {**p, "reset": torch.where(p["reset"] & (marks == 0), 7, marks).to(torch.uint8)}
    out, h_last, ck = torch.full_like(y, 9.0), torch.full_like(last, 9.0), torch.full_like(kept, 9.0)
    for spare in (0, 512):
        need = mamba.gated_scan_fwd_workspace_size(B, D, L) + spare
        ws = torch.full((max(need, 1),), 255, dtype=torch.uint8, device="cuda")
        same = _forward(own, out=out, h_last=h_last, checkpoints=ck, workspace=ws)
        assert same is out
        assert torch.equal(out, y) and torch.equal(h_last, last) and torch.equal(ck, kept)
        need = mamba.gated_scan_bwd_workspace_size(B, D, L) + spare
        ws = torch.full((max(need, 1),), 255, dtype=torch.uint8, device="cuda")
        again = _backward(own, q, checkpoints=ck, workspace=ws)
        assert all(torch.equal(got[n], again[n]) for n in GRADS)
    if mamba.gated_scan_bwd_workspace_size(B, D, L):
        with pytest.raises(mamba.MambaError):
            _backward(own, q, checkpoints=ck, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))

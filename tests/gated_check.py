"""The gated linear recurrence in 64 bits, step by step, with bounds on the error of
a 32-bit evaluation of the same formulas.

Units u = 2^-24 (half a step of fp32), relative unless said otherwise.  The hardware's
2^x, reciprocal, root and reciprocal root are within one step (2 u).
  sigmoid  argument of up to 10 log2 e = 14.4 rounded (14.4 ln2 u), 2^x (2 u), 1 + p (u),
           reciprocal (2 u): below 16 u
  v        the rate (6 u: ln(1 + e^x) and two products), sigmoid, product: below 24 u
  m        half of the error of 1 - a^2 (v's; where it is taken from a, from 2^-v = 0.917
           down, twice a's 2 u of a^2 = 0.84 over 0.16: 22 u) and the root: below 26 u
  input    m, sigmoid, two products: below 44 u of |b|
  a        2^-v: v 24 u absolute from v's error, 3 u of its own
  v dm/dv  v, a^2 (twice a's), 1 / m, sigmoid, products: below (76 + 48 v) u
A step's error is then a times the last one's, 44 u |b|, and (24 v + 4) u a |h|, where h
stands for the recurrence of the absolute values.  Joining spans costs a rounding of its
sums for each of about 20 joins every 8 steps: 3 u a step more.  2^x gives 0 below the normal range, so a is also
off by up to TINY = 2^-126 absolutely, whatever its size."""
import torch

U = 2.0 ** -24
TINY = 2.0 ** -126
HALF_STEP = {torch.float32: U, torch.bfloat16: 2.0 ** -8}


def make(B, D, L, io, seed, gate=True, h0=True, biases=True, reset=0.0, decay=(0.9, 0.999), spread=1.0):
    """Inputs on the CPU; decay: range of a at r = 0."""
    gen = torch.Generator().manual_seed(seed)
    normal = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    p = {"x": normal(B, D, L).to(io), "r": (spread * normal(B, D, L)).to(io), "i": normal(B, D, L).to(io)}
    keep = decay[0] + (decay[1] - decay[0]) * torch.rand(D, generator=gen, dtype=torch.float64)
    p["lam"] = torch.log(torch.expm1(-2.0 * torch.log(keep) / 8.0)).float()
    p["r_bias"] = 0.3 * normal(D) if biases else None
    p["i_bias"] = 0.3 * normal(D) if biases else None
    p["z"] = normal(B, D, L).to(io) if gate else None
    p["h0"] = normal(B, D) if h0 else None
    p["reset"] = torch.rand(B, L, generator=gen) < reset if reset else None
    return p


def gradient_inputs(p, seed, last=True):
    gen = torch.Generator().manual_seed(seed)
    shape = p["x"].shape
    return {"dout": torch.randn(shape, generator=gen).to(p["x"].dtype),
            "dh_last": torch.randn(shape[:2], generator=gen) if last else None}


def _d(t):
    return None if t is None else t.double()


def _parts(p, c):
    x, r, i = _d(p["x"]), _d(p["r"]), _d(p["i"])
    rb = 0.0 if p["r_bias"] is None else _d(p["r_bias"])[:, None]
    ib = 0.0 if p["i_bias"] is None else _d(p["i_bias"])[:, None]
    rate = c * torch.nn.functional.softplus(_d(p["lam"]), threshold=1e4)[:, None]
    sr, si = torch.sigmoid(r + rb), torch.sigmoid(i + ib)
    v = rate * sr
    a, m = torch.exp(-v), torch.sqrt(-torch.expm1(-2.0 * v))
    keeps = v == 0
    first = None if p["reset"] is None else p["reset"].bool()[:, None, :].expand_as(x)
    if first is not None:
        a, m = torch.where(first, 0.0, a), torch.where(first, 1.0, m)
    b = torch.where((m == 0) & torch.isfinite(x), 0.0, m * si * x)
    return x, sr, si, v, a, m, b, first, keeps


def _run(a, b, start, first, reverse=False):
    """s_t = a_t s_(t-1) + b_t in the order of steps, a state dropped at a reset whatever it is."""
    out, s = torch.empty_like(b), start
    steps = range(b.shape[-1] - 1, -1, -1) if reverse else range(b.shape[-1])
    for t in steps:
        moved = a[..., t] * s
        if first is not None:
            moved = torch.where(first[..., t], 0.0, moved)
        s = moved + b[..., t]
        out[..., t] = s
    return out


def forward(p, c=8.0):
    """{"y", "h_last", "h"} and their bounds under "y_err", "h_err"."""
    x, sr, si, v, a, m, b, first, _ = _parts(p, c)
    B, D, L = x.shape
    h0 = torch.zeros(B, D, dtype=torch.float64) if p["h0"] is None else _d(p["h0"])
    h = _run(a, b, h0, first)
    size = _run(a, b.abs(), h0.abs(), first)
    before = torch.cat([h0.abs()[..., None], size[..., :-1]], -1)
    err = _run(a, 44 * U * b.abs() + ((24 * v + 7) * U * a + TINY) * before, torch.zeros_like(h0), first)
    y, y_err = h, err
    if p["z"] is not None:
        z = _d(p["z"])
        silu = z * torch.sigmoid(z)
        y, y_err = h * silu, err * silu.abs() + 20 * U * (h * silu).abs()
    y_err = y_err + HALF_STEP[p["x"].dtype] * (y.abs() + y_err)
    last = h[..., -1] if L else h0
    last_err = err[..., -1] if L else torch.zeros_like(h0)
    return {"y": y, "y_err": y_err + 1e-37, "h": h, "h_last": last, "h_last_err": last_err + 1e-37, "h_err": err,
            "size": size}


def backward(p, q, c=8.0):
    """The gradients and, under name + "_err", their bounds."""
    x, sr, si, v, a, m, b, first, keeps = _parts(p, c)
    B, D, L = x.shape
    io = p["x"].dtype
    zero = torch.zeros(B, D, dtype=torch.float64)
    f = forward(p, c)
    h0 = zero if p["h0"] is None else _d(p["h0"])
    before = torch.cat([h0[..., None], f["h"][..., :-1]], -1)
    before_err = torch.cat([zero[..., None], f["h_err"][..., :-1]], -1)
    dout = _d(q["dout"])
    grad, out = dout, {}
    if p["z"] is not None:
        z = _d(p["z"])
        sz = torch.sigmoid(z)
        grad = dout * z * sz
        slope = sz * (1 + z * (1 - sz))
        # 1 - sigmoid is off by 16 u of 1; z times that, and the products
        out["dz"] = dout * f["h"] * slope
        out["dz_err"] = (dout.abs() * f["h_err"] * slope.abs() +
                         (dout * f["h"]).abs() * sz * (20 * U + z.abs() * 24 * U) + 24 * U * out["dz"].abs())
    end = zero if q["dh_last"] is None else _d(q["dh_last"])
    # what enters from behind is a_(t+1) g_(t+1); behind the last step it is dh_last
    none = torch.zeros(B, D, 1, dtype=torch.bool)
    a_next = torch.cat([a[..., 1:], torch.ones(B, D, 1, dtype=torch.float64)], -1)
    drop_next = None if first is None else torch.cat([first[..., 1:], none], -1)
    v_next = torch.cat([v[..., 1:], zero[..., None]], -1)
    g = _run(a_next, grad, end, drop_next, reverse=True)
    size = _run(a_next, grad.abs(), end.abs(), drop_next, reverse=True)
    behind = torch.cat([size[..., 1:], end.abs()[..., None]], -1)
    g_err = _run(a_next, 20 * U * grad.abs() + ((24 * v_next + 7) * U * a_next + TINY) * behind, zero, drop_next, reverse=True)
    out["dx"], out["di"] = g * m * si, g * m * x * si * (1 - si)
    out["dx_err"] = g_err * m * si + 44 * U * out["dx"].abs()
    out["di_err"] = g_err * (m * x * si * (1 - si)).abs() + (g * m * x).abs() * si * (48 * U)
    ratio = torch.where(m > 0, v * a * a / m.clamp_min(1e-300), 0.0)  # v dm/dv, to 0 with v
    dv_m, dv_a = ratio * si * x, v * a * before
    dq = g * (dv_m - dv_a)
    dq_err = (g_err * (dv_m.abs() + dv_a.abs()) + g.abs() * v * a * before_err +
              g.abs() * (dv_m.abs() + dv_a.abs()) * ((76 + 48 * v) * U) +
              g.abs() * v * TINY * ((si * x).abs() + before.abs()))
    if first is not None:
        dq, dq_err = torch.where(first, 0.0, dq), torch.where(first, 0.0, dq_err)
    dq, dq_err = torch.where(keeps, 0.0, dq), torch.where(keeps, 1e-30, dq_err)
    out["dr"] = dq * (1 - sr)
    out["dr_err"] = dq_err * (1 - sr) + dq.abs() * 18 * U
    for name in [n for n in ("dx", "dr", "di", "dz") if n in out]:
        out[name + "_err"] += HALF_STEP[io] * (out[name].abs() + out[name + "_err"]) + 1e-37
    lam = _d(p["lam"])
    scale = torch.sigmoid(lam) / torch.nn.functional.softplus(lam, threshold=1e4)
    depth = (L // 64 + 24 + B) * U  # roundings on a term's way through a lane, its wave and the batch
    total = lambda t: t.sum(dim=(0, 2))  # noqa: E731
    unrounded = {"dr": dq_err * (1 - sr) + dq.abs() * 18 * U, "di": g_err * (m * x * si * (1 - si)).abs() +
                 (g * m * x).abs() * si * (48 * U)}
    out["dlam"] = total(dq) * scale
    out["dlam_err"] = (total(dq_err) + depth * total(dq.abs())) * scale + 16 * U * out["dlam"].abs() + 1e-37
    for name, of in (("dr_bias", "dr"), ("di_bias", "di")):
        out[name] = total(out[of])
        out[name + "_err"] = total(unrounded[of]) + depth * total(out[of].abs()) + 1e-37
    out["dh0"] = end.clone() if L == 0 else a[..., 0] * g[..., 0]
    out["dh0_err"] = torch.zeros_like(end) + 1e-37
    if L:
        if first is not None:
            out["dh0"] = torch.where(first[..., 0], 0.0, out["dh0"])
        out["dh0_err"] = out["dh0_err"] + a[..., 0] * g_err[..., 0] + ((24 * v[..., 0] + 7) * U * a[..., 0] + TINY) * size[..., 0]
    return out


def worst(got, want, err):
    """The largest part of its bound that an element's error takes; NaN has to meet NaN."""
    got = got.double().cpu()
    assert got.shape == want.shape, (got.shape, want.shape)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), "NaN in other places"
    if got.numel() == 0:
        return 0.0
    part = (got - want).abs() / err
    return part[~torch.isnan(want)].max().item() if (~torch.isnan(want)).any() else 0.0

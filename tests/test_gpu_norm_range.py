"""GPU parity of the residual RMS norm and its gradient with the formulas in 64
bits on rows whose sum of squares leaves the fp32 range on either side, beside
ordinary rows (of the same wave where a wave has several), and on zero rows
without eps.

Tolerances, from the arithmetic (u = 2^-24).  A lane adds the 8 squares of a
chunk one by one, then the sums of up to 8 chunks; 6 steps over the lanes and 16
over the waves follow: with the product, a sum of squares is below 1 + 8 + 8 + 6
+ 16 = 39 u relative, the mean with eps below 41 u, 1/sqrt of it below 21 + 2 u,
y = h r w below 27 u: SUM = 4e-6 (67 u) of |y| holds.  dh = r (w dy - (h r) r
mean(w dy h)) has r twice (46 u), the sum (40 u of the sum of magnitudes) and 6
products: below 95 u of the terms' magnitudes, GRAD = 1.2e-5 (200 u); dweight
adds r h dy (25 u) of up to 129 rows and then the groups, below 100 u more.  Taking rows by powers of two adds nothing."""
import pytest

from scan_check import say

pytestmark = pytest.mark.gpu

SUM, GRAD, HALF_BF16 = 4e-6, 1.2e-5, 2.0 ** -8
WIDTHS = [1, 5, 8, 60, 100, 200, 500, 771, 1024, 1500, 2560, 4100, 9000, 20000, 32768]


def _t(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def _rows(M, D, io, seed, scales):
    """Row m is of size scales[m % len(scales)]."""
    import torch
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((M, D), generator=g).double().clamp(-3, 3)
    size = torch.tensor(scales, dtype=torch.float64)[torch.arange(M) % len(scales)]
    return (x * size[:, None]).to(_t(io)).cuda()


def _norm64(h, w, eps):
    import torch
    size = (h.square().mean(-1, keepdim=True) + eps).sqrt()
    return torch.where(size > 0, h / size, torch.zeros_like(h)) * w.double()  # zero rows without eps: zeros


# Sizes from near the smallest number to near the largest, and none at all.
SCALES = [1.0, 1e25, 1e-25, 0.0, 3e18, 1e-19, 9e37, 1e-41, 2.5]


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("io,res", [("f32", None), ("f32", "f32"), ("bf16", None), ("bf16", "f32"),
                                    ("bf16", "bf16")])
def test_norm(D, io, res):
    import torch
    import selective_state_space_80_amd as mamba
    for M in (9, 1030) if D <= 2560 else (9,):
        for eps in (0.0, 1e-30, 1e-5):
            x = _rows(M, D, io, D, SCALES)
            r = None if res is None else _rows(M, D, res, D + 1, [0.0] if res == "bf16" else SCALES)
            w = 1.0 + 0.1 * torch.randn((D,), generator=torch.Generator().manual_seed(D + 2)).cuda()
            h32 = x.float() if r is None else x.float() + r.float()
            y = _norm64(h32.double(), w, eps)
            got = mamba.rms_norm(x, w, residual=r, eps=eps)
            out, kept = (got, None) if r is None else got
            fine = torch.isfinite(h32).all(-1)  # the sum itself may pass the range
            assert torch.equal(torch.isfinite(out).all(-1), fine), (M, D, eps)
            tol = SUM + (HALF_BF16 if io == "bf16" else 0.0)
            assert bool(((out.double() - y).abs() <= tol * y.abs() + 1e-37)[fine].all()), (M, D, eps)
            if r is not None:
                assert torch.equal(kept, h32.to(kept.dtype)), (M, D, eps)
            q, s, *_ = mamba.rms_norm_int8(x, w, residual=r, eps=eps)
            assert torch.equal(torch.isfinite(s), fine) and not q[~fine].any()
            q, s, y = q[fine], s[fine], y[fine]
            top = y.abs().amax(-1)
            assert bool(((s.double() - top / 127).abs() <= (SUM + 2.0 ** -23) * top / 127 + 1e-37).all()), (M, D, eps)
            steps = torch.where(top > 0, 127.0 / top.clamp_min(1e-300), torch.zeros_like(top))
            off = (q.double() - y * steps[:, None]).abs()
            # rows whose norm is itself next to the smallest number (a small row
            # under a large eps) keep few bits of it
            assert bool((off[top > 1e-30] <= 0.5 + 127 * 2 * SUM).all()), (M, D, eps)
            assert not q[top == 0].any()
    say(f"norm range D={D} {io} {res} ok")


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("io,hio", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("given", [False, True])
def test_gradient(D, io, hio, given):
    import torch
    import selective_state_space_80_amd as mamba
    scales = [1.0, 1e25, 1e-25, 0.0, 3e18, 1e-19, 9e37, 2.5]
    for M in (8, 1030) if D <= 2560 else (8,):
        for eps in (0.0, 1e-5):
            h = _rows(M, D, hio, D + 3, scales)
            dy = _rows(M, D, io, D + 4, [1.0])
            dres = _rows(M, D, hio, D + 5, [1.0, 1e-25, 1e25]) if given else None
            w = 1.0 + 0.1 * torch.randn((D,), generator=torch.Generator().manual_seed(D + 6)).cuda()
            hd, gd, wd = h.double(), dy.double(), w.double()
            size = (hd.square().mean(-1, keepdim=True) + eps).sqrt()
            r = torch.where(size > 0, 1.0 / size, torch.zeros_like(size))  # zero rows: no gradient through the norm
            n = hd * r
            along = wd * gd * n
            dh = r * (wd * gd - n * along.mean(-1, keepdim=True))
            bound = r * ((wd * gd).abs() + n.abs() * along.abs().mean(-1, keepdim=True))
            if given:
                dh, bound = dh + dres.double(), bound + dres.double().abs()
            g = mamba.rms_norm_bwd(dy, h, w, dresidual_out=dres, eps=eps)
            half = HALF_BF16 * dh.abs() if io == "bf16" else 0.0
            assert bool(((g["dx"].double() - dh).abs() <= GRAD * bound + half + 1e-37).all()), (M, D, eps, "dx")
            if hio != io:
                assert bool(((g["dresidual"].double() - dh).abs() <= GRAD * bound + 1e-37).all()), (M, D, eps)
            terms = gd * n
            assert bool(((g["dweight"].double() - terms.sum(0)).abs() <= GRAD * terms.abs().sum(0) + 1e-37).all()), (M, D)
    say(f"gradient range D={D} {io} {hio} ok")


@pytest.mark.parametrize("D", [1, 7, 300, 2560])
def test_rows_that_are_not_finite_stay_so(D):
    import torch
    import selective_state_space_80_amd as mamba
    x = _rows(6, D, "f32", D, [1.0, 1e25])
    x[2, D - 1], x[3, 0] = float("inf"), float("nan")
    q, s = mamba.rms_norm_int8(x, torch.ones(D, device="cuda"), eps=0.0)
    assert torch.isnan(s).tolist() == [False, False, True, True, False, False] and not q[2:4].any()
    out = mamba.rms_norm(x, torch.ones(D, device="cuda"), eps=0.0)
    assert torch.isnan(out[2, D - 1]) and torch.isnan(out[3]).all() and torch.isfinite(out[[0, 1, 4, 5]]).all()

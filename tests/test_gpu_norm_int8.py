"""GPU parity of the residual RMS norm (plain and 8-bit output), its gradient
and the 8-bit quantiser with their formulas in 64 bits.

Tolerances, from the arithmetic (u = 2^-24, fp32 rounding; bf16 outputs add
half an ulp, at most 2^-8 relative):
  sums over a row add at most 32 elements in a lane, then 6 + 16 partial sums:
  relative error of a sum of squares below 64 u, of r = 1/sqrt below 36 u, of
  y = h r w below 40 u: SUM = 4e-6 (= 67 u) of |y|.  dh has r^3 (below 110 u)
  and the sum of w dy h (64 u of the sum of magnitudes): GRAD = 1.2e-5 (= 200 u)
  of its terms' magnitudes; dweight likewise of the sum of |dy h r| (at most 100
  additions in a row at these sizes).  The quantiser's scale is one division
  (u), and v * mul is off by 2u * 127 of a step before it is rounded."""
import numpy as np
import pytest

from scan_check import say

pytestmark = pytest.mark.gpu

SUM, GRAD, HALF_BF16 = 4e-6, 1.2e-5, 2.0 ** -8
TYPES = ["f32", "bf16"]


def _t(name):
    import torch
    return {"f32": torch.float32, "bf16": torch.bfloat16}[name]


def _draw(shape, io, seed, scale=1.0):
    import torch
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(_t(io)).cuda()


def _norm64(x, res, w, eps):
    h = x.double() if res is None else x.double() + res.double()
    r = 1.0 / (h.square().mean(-1, keepdim=True) + eps).sqrt()
    return h, r, h * r * w.double()


def _close(got, want, tol, what, size=None):
    """|got - want| <= tol * size (size: |want| unless given)."""
    import torch
    assert got.shape == want.shape, what
    bound = tol * (want.abs() if size is None else size) + 1e-37
    err = (got.double() - want).abs()
    assert bool(torch.isfinite(got.double()).all()), what
    worst = (err / bound).max().item() if err.numel() else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3f} of the bound"
    return worst


def _out_tol(io, tol):
    return tol + (HALF_BF16 if io == "bf16" else 0.0)


def _check_int8(q, scale, y, slack, what):
    """q and scale against the 64-bit rows y whose own error is slack * |y|."""
    import torch
    top = y.abs().amax(-1)
    _close(scale, top / 127.0, slack + 2.0 ** -23, what + " scale")
    steps = torch.where(top > 0, 127.0 / top.clamp_min(1e-300), torch.zeros_like(top))
    off = (q.double() - y * steps.unsqueeze(-1)).abs().max().item() if q.numel() else 0.0
    assert q.dtype == torch.int8 and int(q.to(torch.int32).abs().max()) <= 127
    assert off <= 0.5 + 127 * (2 * slack + 2.0 ** -23), f"{what}: q off by {off}"


WIDTHS = [1, 3, 7, 8, 9, 64, 100, 511, 512, 513, 768, 771, 1032, 1500, 2560, 2567, 4096, 4104, 5120, 8192,
          16391, 32768]


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("io,res", [("f32", None), ("f32", "f32"), ("bf16", None), ("bf16", "f32"),
                                    ("bf16", "bf16")])
def test_norm(D, io, res):
    import torch
    import selective_state_space_80_amd as mamba
    eps = 1e-5
    for M in ([1, 6, 1027] if D <= 5120 else [1, 6]):
        x = _draw((M, D), io, 1 + D)
        r = None if res is None else _draw((M, D), res, 2 + D, 3.0)
        w = 1.0 + 0.1 * _draw((D,), "f32", 3 + D)
        h, _, y = _norm64(x, r, w, eps)
        got = mamba.rms_norm(x, w, residual=r, eps=eps)
        out, kept = (got, None) if res is None else got
        _close(out, y, _out_tol(io, SUM), f"norm M={M} D={D} {io} {res}")
        q, s, *kept8 = mamba.rms_norm_int8(x, w, residual=r, eps=eps)
        _check_int8(q, s, y, SUM, f"norm int8 M={M} D={D} {io} {res}")
        if res is not None:
            _close(kept, h, _out_tol(res, 2.0 ** -24), "residual_out")
            assert torch.equal(kept8[0], kept)
            # in place: the same bits, in the residual's own buffer
            own = r.clone()
            out2, kept2 = mamba.rms_norm(x, w, residual=own, eps=eps, residual_out=own)
            assert kept2 is own and torch.equal(own, kept) and torch.equal(out2, out)
            own = r.clone()
            q2, s2, _ = mamba.rms_norm_int8(x, w, residual=own, eps=eps, residual_out=own)
            assert torch.equal(own, kept) and torch.equal(q2, q) and torch.equal(s2, s)
    say(f"norm D={D} {io} {res} ok")


@pytest.mark.parametrize("D", [1, 5, 8, 12, 63, 100, 512, 771, 1024, 1025, 2560, 4100, 5120, 8195, 32768])
@pytest.mark.parametrize("io,hio", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("given", [False, True])
def test_norm_gradient(D, io, hio, given):
    import torch
    import selective_state_space_80_amd as mamba
    eps = 1e-5
    for M in ([1, 5, 2063] if D <= 2560 else [1, 9]):
        h = _draw((M, D), hio, 11 + D, 2.0)
        dy = _draw((M, D), io, 12 + D)
        dres = _draw((M, D), hio, 13 + D) if given else None
        w = 1.0 + 0.1 * _draw((D,), "f32", 14 + D)
        hd, gd, wd = h.double(), dy.double(), w.double()
        r = 1.0 / (hd.square().mean(-1, keepdim=True) + eps).sqrt()
        along = wd * gd * hd
        dh = r * wd * gd - r ** 3 * hd * along.mean(-1, keepdim=True)
        size = (r * wd * gd).abs() + r ** 3 * hd.abs() * along.abs().mean(-1, keepdim=True)
        if given:
            dh, size = dh + dres.double(), size + dres.double().abs()
        g = mamba.rms_norm_bwd(dy, h, w, dresidual_out=dres, eps=eps)
        half = HALF_BF16 * dh.abs()
        err = (g["dx"].double() - dh).abs()
        assert (err <= GRAD * size + (half if io == "bf16" else 0.0) + 1e-37).all(), (M, D, "dx")
        assert g["dx"].dtype == dy.dtype and g["dresidual"].dtype == h.dtype
        if hio != io:
            err = (g["dresidual"].double() - dh).abs()
            assert (err <= GRAD * size + 1e-37).all(), (M, D, "dresidual")
        else:
            assert g["dresidual"] is g["dx"]
        terms = gd * hd * r
        _close(g["dweight"], terms.sum(0), GRAD, "dweight", terms.abs().sum(0))
        again = mamba.rms_norm_bwd(dy, h, w, dresidual_out=dres, eps=eps)
        assert all(torch.equal(g[k], again[k]) for k in g)  # fixed order of the sums
    say(f"norm gradient D={D} {io} {hio} ok")


def test_norm_gradient_against_differences():
    """Central differences, in 64 bits, of J = sum(y dy) + sum(h dres)."""
    import torch
    import selective_state_space_80_amd as mamba
    M, D, eps, step = 3, 21, 1e-5, 1e-5
    h, dy = _draw((M, D), "f32", 31), _draw((M, D), "f32", 32)
    dres, w = _draw((M, D), "f32", 33), 1.0 + 0.1 * _draw((D,), "f32", 34)

    def J(hd, wd):
        y = hd / (hd.square().mean(-1, keepdim=True) + eps).sqrt() * wd
        return (y * dy.double()).sum() + (hd * dres.double()).sum()

    g = mamba.rms_norm_bwd(dy, h, w, dresidual_out=dres, eps=eps)
    hd, wd = h.double(), w.double()
    for i in range(M):
        for j in range(D):
            e = torch.zeros_like(hd)
            e[i, j] = step
            want = ((J(hd + e, wd) - J(hd - e, wd)) / (2 * step)).item()
            assert abs(g["dx"][i, j].item() - want) <= 5e-5, (i, j)
    for j in range(D):
        e = torch.zeros_like(wd)
        e[j] = step
        want = ((J(hd, wd + e) - J(hd, wd - e)) / (2 * step)).item()
        assert abs(g["dweight"][j].item() - want) <= 5e-5, j


@pytest.mark.parametrize("D", [5, 60, 700, 2560, 9000, 20000])
def test_norm_gradient_of_small_rows(D):
    """Rows so small that 1/rms has no cube in fp32, and zero rows beside them."""
    import torch
    import selective_state_space_80_amd as mamba
    M, eps = 6, 1e-29
    h, dy = _draw((M, D), "f32", 35 + D, 1e-14), _draw((M, D), "f32", 36 + D)
    h[2] = 0.0
    w = 1.0 + 0.1 * _draw((D,), "f32", 37 + D)
    g = mamba.rms_norm_bwd(dy, h, w, eps=eps)
    hd, gd, wd = h.double(), dy.double(), w.double()
    r = 1.0 / (hd.square().mean(-1, keepdim=True) + eps).sqrt()
    along = wd * gd * hd
    dh = r * wd * gd - r ** 3 * hd * along.mean(-1, keepdim=True)
    size = (r * wd * gd).abs() + r ** 3 * hd.abs() * along.abs().mean(-1, keepdim=True)
    assert ((g["dx"].double() - dh).abs() <= GRAD * size + 1e-37).all()
    terms = gd * hd * r
    _close(g["dweight"], terms.sum(0), GRAD, "dweight", terms.abs().sum(0))


def test_norm_gradient_of_nothing():
    import torch
    import selective_state_space_80_amd as mamba
    g = mamba.rms_norm_bwd(torch.empty((0, 100), device="cuda"), torch.empty((0, 100), device="cuda"),
                           torch.ones(100, device="cuda"))
    assert g["dx"].shape == (0, 100) and torch.equal(g["dweight"], torch.zeros(100, device="cuda"))
    w = torch.ones(16, device="cuda")
    assert mamba.rms_norm(torch.empty((0, 16), device="cuda"), w).shape == (0, 16)
    q, s = mamba.rms_norm_int8(torch.empty((2, 0, 16), device="cuda"), w)
    assert q.shape == (2, 0, 16) and s.shape == (2, 0)


@pytest.mark.parametrize("K", WIDTHS)
@pytest.mark.parametrize("io", TYPES)
def test_quantize_tokens(K, io):
    import torch
    import selective_state_space_80_amd as mamba
    for M in ([1, 7, 1030] if K <= 5120 else [1, 7]):
        x = _draw((M, K), io, 41 + K, 5.0)
        q, s = mamba.quantize_int8(x)
        _check_int8(q, s, x.double(), 0.0, f"quantize M={M} K={K} {io}")
        # correctly rounded (through fp64: torch's own fp32 form multiplies by 1/127)
        assert torch.equal(s, (x.double().abs().amax(-1) / 127.0).float())


@pytest.mark.parametrize("B,K,L", [(1, 1, 1), (2, 3, 5), (1, 64, 64), (3, 65, 63), (1, 128, 256), (2, 771, 130),
                                   (1, 5120, 200), (2, 1536, 1), (1, 7, 1001), (1, 40000, 33), (2, 2568, 96),
                                   (1, 8192, 72)])
@pytest.mark.parametrize("io", TYPES)
def test_quantize_channel_major(B, K, L, io):
    """Channel-major input gives the bits of the token-major call on its transpose."""
    import torch
    import selective_state_space_80_amd as mamba
    x = _draw((B, K, L), io, 51 + K, 2.0)
    q, s = mamba.quantize_int8(x, channel_major=True)
    y = x.transpose(1, 2).contiguous()
    _check_int8(q, s, y.double(), 0.0, f"quantize channel-major {B} {K} {L} {io}")
    if K <= 32768:
        q2, s2 = mamba.quantize_int8(y)
        assert torch.equal(q, q2) and torch.equal(s, s2)


@pytest.mark.parametrize("L", [2, 3, 4, 5, 6, 7])
@pytest.mark.parametrize("B,K", [(1, 1), (3, 4), (2, 5), (4, 259), (2, 4093), (130, 1536), (2, 5120), (1, 8201),
                                 (1, 40001)])
@pytest.mark.parametrize("io", TYPES)
def test_quantize_channel_major_of_few_tokens(B, K, L, io):
    import torch
    import selective_state_space_80_amd as mamba
    x = _draw((B, K, L), io, 52 + K + L, 2.0)
    q, s = mamba.quantize_int8(x, channel_major=True)
    y = x.transpose(1, 2).contiguous()
    _check_int8(q, s, y.double(), 0.0, f"quantize channel-major {B} {K} {L} {io}")
    if K <= 32768:
        q2, s2 = mamba.quantize_int8(y)
        assert torch.equal(q, q2) and torch.equal(s, s2)


@pytest.mark.parametrize("B,K,L", [(40, 100, 3), (40, 5000, 5), (3, 9001, 6), (200, 70, 9), (200, 1030, 21),
                                   (3, 6145, 100), (2, 8192, 515), (2, 12289, 75), (1, 20000, 130),
                                   (1, 24577, 70), (2, 32768, 33)])
@pytest.mark.parametrize("io", TYPES)
def test_quantize_channel_major_special_tokens(B, K, L, io):
    """Tokens of zeros, of the smallest numbers, and with a NaN or an infinity
    anywhere, among ordinary ones, in every tiling: the bits of the token-major call."""
    import torch
    import selective_state_space_80_amd as mamba
    y = _draw((B * L, K), io, 53 + K + L)
    n = torch.arange(B * L, device="cuda")
    y[n % 11 == 1] = 0.0
    y[n % 11 == 3] *= 1e-38
    y[n % 11 == 5, K - 1] = float("nan")
    y[n % 11 == 7, K // 3] = float("inf")
    y[n % 11 == 9] = torch.finfo(_t(io)).min
    y = y.view(B, L, K)
    q, s = mamba.quantize_int8(y.transpose(1, 2).contiguous(), channel_major=True)
    q2, s2 = mamba.quantize_int8(y)
    assert torch.equal(q, q2) and torch.equal(s.view(torch.int32), s2.view(torch.int32))


@pytest.mark.parametrize("K", [5, 100, 2560, 6000])
@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("form", ["token", "channel", "norm"])
def test_special_rows(K, io, form):
    """Zero rows, rows of the type's lowest value, rows near the smallest
    numbers, and rows that hold a NaN or an infinity anywhere."""
    import torch
    import selective_state_space_80_amd as mamba
    inf, nan = float("inf"), float("nan")
    rows = _draw((10, K), io, 61 + K)
    rows[1] = 0.0
    rows[2, K - 1] = nan
    rows[3, 0] = inf
    rows[4, K // 2] = -inf
    rows[5] = rows[5] * 1e-38
    rows[6] = torch.finfo(_t(io)).min
    rows[7] = 0.0
    rows[7, K - 1] = -3.0
    rows[8] = -0.0
    if form == "norm":
        w = torch.ones(K, device="cuda")
        rows[5], rows[6] = 1e-6, 1e3  # the square sum is an fp32 sum
        q, s = mamba.rms_norm_int8(rows, w, eps=1e-12)
    elif form == "token":
        q, s = mamba.quantize_int8(rows)
    else:
        q, s = mamba.quantize_int8(rows.t().contiguous()[None], channel_major=True)
        q, s = q[0], s[0]
    for i in (2, 3, 4):
        assert torch.isnan(s[i]) and not q[i].any(), i
    for i in (1, 8):
        assert s[i] == 0 and not q[i].any(), i
    fine = torch.tensor([0, 7, 9], device="cuda")
    y = rows[fine].double()
    if form == "norm":
        y = _norm64(rows[fine], None, w, 1e-12)[2]
    _check_int8(q[fine], s[fine], y, SUM, "ordinary rows beside special ones")
    assert (q[6].to(torch.int32).abs() == 127).all()
    if form == "norm":
        assert (q[5] == 127).all()
    else:  # the integers are right although 127 / max|x| passes the fp32 range
        v = rows[5].double()
        want = v * (127.0 / v.abs().max())
        assert (q[5].double() - want).abs().max() <= 0.5 + 1e-4
        assert torch.equal(s[6], (rows[6].double().abs().max() / 127.0).float())


@pytest.mark.parametrize("M,D", [((1 << 22) + 5, 40), (70000, 32768)])
def test_many_rows_and_offsets_past_32_bits(M, D):
    """More rows than 2^22, and tensors of more than 2^31 elements."""
    import torch
    import selective_state_space_80_amd as mamba
    x = _draw((1, D), "bf16", 81).expand(M, D).contiguous()
    x[-1] = _draw((D,), "bf16", 82)
    x[M // 2] = 0.0
    w = 1.0 + 0.1 * _draw((D,), "f32", 83)
    rows = torch.tensor([0, 1, M // 2 - 1, M // 2, M // 2 + 1, M - 2, M - 1], device="cuda")
    y = _norm64(x[rows], None, w, 1e-5)[2]
    q, s = mamba.rms_norm_int8(x, w)
    _check_int8(q[rows], s[rows], y, SUM, "norm int8")
    del q
    q, s = mamba.quantize_int8(x)
    _check_int8(q[rows], s[rows], x[rows].double(), 0.0, "quantize")
    del q
    out = mamba.rms_norm(x, w)
    _close(out[rows], y, _out_tol("bf16", SUM), "norm")
    del out
    if D <= 4096:
        g = mamba.rms_norm_bwd(x, x, w)
        h = x[rows].double()
        r = 1.0 / (h.square().mean(-1, keepdim=True) + 1e-5).sqrt()
        along = (w.double() * h * h).mean(-1, keepdim=True)
        dh = r * w.double() * h - r ** 3 * h * along
        size = (r * w.double() * h).abs() + r ** 3 * h.abs() * along.abs()
        err = (g["dx"][rows].double() - dh).abs()
        assert (err <= GRAD * size + HALF_BF16 * dh.abs() + 1e-37).all()
    torch.cuda.empty_cache()


def test_channel_major_offsets_past_32_bits():
    import torch
    import selective_state_space_80_amd as mamba
    K, L = 5120, 440000
    x = torch.empty((1, K, L), dtype=torch.bfloat16, device="cuda")
    x[:] = _draw((1, K, 1), "bf16", 84)
    x[0, K - 1, L - 1] = 1000.0
    q, s = mamba.quantize_int8(x, channel_major=True)
    for l in (0, 1, L // 2, L - 2, L - 1):
        _check_int8(q[0, l], s[0, l:l + 1].squeeze(), x[0, :, l].double(), 0.0, f"token {l}")
    del x, q
    torch.cuda.empty_cache()


def test_unaligned_storage():
    """Rows that start at any element of their storage."""
    import torch
    import selective_state_space_80_amd as mamba
    for io in TYPES:
        for D in (9, 600, 2561):
            flat = _draw((4 * D + 3,), io, 71 + D)
            x = flat[1:1 + 4 * D].view(4, D)
            r = flat[3:3 + 4 * D].view(4, D)
            w = _draw((D + 1,), "f32", 72)[1:]
            out, kept = mamba.rms_norm(x, w, residual=r)
            want, wkept = mamba.rms_norm(x.clone(), w.clone(), residual=r.clone())
            assert torch.equal(out, want) and torch.equal(kept, wkept)
            q, s = mamba.quantize_int8(x)
            q2, s2 = mamba.quantize_int8(x.clone())
            assert torch.equal(q, q2) and torch.equal(s, s2)
            g = mamba.rms_norm_bwd(x, r, w)
            g2 = mamba.rms_norm_bwd(x.clone(), r.clone(), w.clone())
            assert torch.equal(g["dx"], g2["dx"]) and torch.equal(g["dweight"], g2["dweight"])


def test_refusals():
    import torch
    import selective_state_space_80_amd as mamba
    x, w = torch.zeros((4, 32), device="cuda"), torch.ones(32, device="cuda")
    with pytest.raises(ValueError):
        mamba.rms_norm(x, w[:31].contiguous())
    with pytest.raises(ValueError):
        mamba.rms_norm(x.t(), torch.ones(4, device="cuda"))
    with pytest.raises(ValueError):
        mamba.rms_norm(x, w, residual_out=x)
    with pytest.raises(TypeError):
        mamba.rms_norm(x, w, residual=x.bfloat16())
    with pytest.raises(TypeError):
        mamba.rms_norm(x.half(), w)
    with pytest.raises(TypeError):
        mamba.rms_norm(x, w.bfloat16())
    for bad in (dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf"))):
        with pytest.raises(mamba.MambaError):
            mamba.rms_norm(x, w, **bad)
    with pytest.raises(mamba.MambaError):
        mamba.rms_norm(x, w, out=x)
    with pytest.raises(mamba.MambaError):
        mamba.rms_norm(x, w, residual=x.clone(), residual_out=x)
    with pytest.raises(mamba.MambaError):
        mamba.rms_norm(torch.zeros((1, 40000), device="cuda"), torch.ones(40000, device="cuda"))
    with pytest.raises(mamba.MambaError):
        mamba.quantize_int8(torch.zeros((3, 0), device="cuda"))
    with pytest.raises(TypeError):
        mamba.rms_norm_bwd(x, x.bfloat16(), w)
    with pytest.raises(mamba.MambaError):
        mamba.rms_norm_bwd(x, x.clone(), w, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        mamba.rms_norm(x.cpu(), w.cpu())
